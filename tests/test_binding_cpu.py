"""The binding's own checks, on stand-ins for GPU tensors (CPU only: no call here reaches the library's kernels)."""
import pytest
import torch

import load_balancing_amd as mx


class OnGpu:
    """What the binding asks of a tensor on the current GPU."""

    def __init__(self, numel, dtype, device=0):
        self._numel, self.dtype, self._device = numel, dtype, device
        self.is_cuda, self.device = True, f"cuda:{device}"

    def numel(self):
        return self._numel

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def one_gpu(monkeypatch):
    monkeypatch.setattr(mx, "_current_device", lambda: 0)
    monkeypatch.setattr(mx, "_stream", lambda stream: 0)


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the library's calls, each of which succeeds without doing anything."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(mx, "lib", Library)
    return made


def test_quant_weights_takes_bf16(one_gpu, calls):
    """bf16 values (or their bits, as every bf16 argument): other types of the same size are not read as bf16."""
    E, out, inp = 2, 128, 256
    n = out * inp
    w8 = OnGpu(E * (n + 16), torch.uint8)
    call = lambda w: mx.moonep_quant_weights(mx.Shape(1, E, 0, 1, 16), inp, out, w, n, 0, w8, n + 16, 0, n)  # noqa: E731
    for t in (torch.bfloat16, torch.int16):
        call(OnGpu(E * n, t))
    assert [c[0] for c in calls] == ["moonep_quant_weights"] * 2
    for w in (OnGpu(E * n, torch.float16), OnGpu(E * n // 2, torch.float32), OnGpu(2 * E * n, torch.uint8),
              OnGpu(2 * E * n, torch.float8_e4m3fn)):
        with pytest.raises(ValueError, match="dtype"):
            call(w)
    with pytest.raises(ValueError, match="elements"):
        call(OnGpu(E * n - 8, torch.bfloat16))
    assert len(calls) == 2


@pytest.mark.parametrize("internal", [True, False], ids=["internal", "public"])
def test_current_stream(monkeypatch, internal):
    """The current stream of the current device, also from a torch without its internal accessor of the handle."""

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    if internal:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 70 + device, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert mx._stream(None) == (73 if internal else 77)
    assert mx._stream(5) == 5 and mx._stream(Stream()) == 77
