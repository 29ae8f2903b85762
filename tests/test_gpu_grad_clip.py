"""The gradients' norm and clipping on an MI355X, against fp64."""
import math

import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def tensors(sizes, types, g, std=1.0):
    """Gradients at odd places of larger buffers, and outputs at other odd places."""
    src, dst = [], []
    for i, (n, t) in enumerate(zip(sizes, types)):
        pad = torch.randn(n + 16, generator=g, device="cuda") * std
        src.append(pad.to(t)[i % 5:i % 5 + n])
        dst.append(torch.full((n + 16,), 5.0, device="cuda", dtype=t)[(3 * i) % 7:(3 * i) % 7 + n])
    return src, dst


SIZES = [
    [1], [7], [8], [4096], [16383, 16384, 16385], [0, 3, 0, 5], [50000, 1, 2, 3, 70001],
    [2049] * 40, [131072 * 3 + 5, 9],
]


def work():
    return torch.full((mx.GRAD_WORKSPACE_BYTES,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("kinds", [(torch.float32,), (torch.bfloat16,), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("ratio", [0.5, 3.0])
def test_norm_and_clip(gpu_ready, sizes, kinds, ratio):
    g = gen()
    types = [kinds[i % len(kinds)] for i in range(len(sizes))]
    src, dst = tensors(sizes, types, g)
    was = [t.clone() for t in src]
    table = mx.moonep_grad_table(src, dst)
    sumsq = sum(float((t.double() ** 2).sum()) for t in src)
    total = math.sqrt(sumsq)
    norm, ss = torch.empty(1, device="cuda"), torch.empty(1, device="cuda", dtype=torch.float64)
    mx.moonep_grad_norm(table, norm, work(), ss)
    # fp64 sums: far below fp32's rounding of the root
    assert abs(ss.item() - sumsq) <= 1e-12 * sumsq
    assert abs(norm.item() - total) <= (2.0 ** -24 + 1e-12) * total
    for given in (None, ss):
        norm.fill_(-1)
        mx.moonep_grad_clip(table, total / ratio, norm, None if given is not None else work(), given)
        assert abs(norm.item() - total) <= (2.0 ** -24 + 1e-12) * total
        f = 1.0 / max(1.0, ratio)
        for t, o, w in zip(src, dst, was):
            assert torch.equal(t, w)
            want = w.double() * f
            # the factor and the product in fp32, one rounding to the type
            half = 2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0
            assert ((o.double() - want).abs() <= (half + 2.0 ** -23 + 1e-12) * want.abs() + 2.0 ** -149).all()
            if ratio < 1:
                assert torch.equal(o, w)
            o.fill_(5.0)


def test_only_the_outputs_are_written(gpu_ready):
    g = gen(1)
    whole = torch.full((3000,), 5.0, device="cuda")
    a, b = torch.randn(700, generator=g, device="cuda"), torch.randn(1001, generator=g, device="cuda")
    table = mx.moonep_grad_table([a, b], [whole[1:701], whole[1003:2004]])
    mx.moonep_grad_clip(table, 0.25, torch.empty(1, device="cuda"), work())
    assert whole[0] == 5 and (whole[701:1003] == 5).all() and (whole[2004:] == 5).all()
    assert not (whole[1:701] == 5).any()


def test_in_place_and_untouched_below_the_limit(gpu_ready):
    g = gen(2)
    a = torch.randn(33333, generator=g, device="cuda")
    b = torch.randn(4444, generator=g, device="cuda").bfloat16()
    table, norm = mx.moonep_grad_table([a, b]), torch.empty(1, device="cuda")
    a0, b0 = a.clone(), b.clone()
    mx.moonep_grad_clip(table, 1e9, norm, work())
    assert torch.equal(a, a0) and torch.equal(b, b0)
    total = norm.item()
    mx.moonep_grad_clip(table, total / 8, norm, work())
    f = torch.tensor((total / 8) / math.sqrt(float((a0.double() ** 2).sum() + (b0.double() ** 2).sum()))).float()
    assert ((a - a0 * f.cuda()).abs() <= 2.0 ** -22 * a0.abs()).all()
    mx.moonep_grad_norm(table, norm, work())
    assert abs(norm.item() - total / 8) <= 1e-3 * total / 8


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_leaves_the_gradients(gpu_ready, bad):
    a = torch.ones(20000, device="cuda")
    a[17777] = bad
    b = torch.full((5,), 2.0, device="cuda").bfloat16()
    a0, norm = a.clone(), torch.empty(1, device="cuda")
    mx.moonep_grad_clip(mx.moonep_grad_table([a, b]), 0.1, norm, work())
    assert not math.isfinite(norm.item())
    assert torch.equal(a.nan_to_num(7.0), a0.nan_to_num(7.0)) and (b == 2).all()


def test_extremes(gpu_ready):
    """Squares beyond fp32 and below it; a limit of 0; zeros; no tensors."""
    norm = torch.empty(1, device="cuda")
    a = torch.full((100,), 2.0 ** 120, device="cuda")
    mx.moonep_grad_clip(mx.moonep_grad_table([a]), 1.0, norm, work())
    assert norm.item() == 10 * 2.0 ** 120 and ((a - 0.1).abs() <= 2.0 ** -24).all()
    a = torch.full((100,), 2.0 ** -100, device="cuda")
    mx.moonep_grad_norm(mx.moonep_grad_table([a]), norm, work())
    assert norm.item() == 10 * 2.0 ** -100
    mx.moonep_grad_clip(mx.moonep_grad_table([a]), 0.0, norm, work())
    assert (a == 0).all()
    mx.moonep_grad_clip(mx.moonep_grad_table([a]), 0.0, norm, work())
    assert norm.item() == 0 and (a == 0).all()
    for none in ([], [torch.empty(0, device="cuda")]):
        norm.fill_(3)
        mx.moonep_grad_clip(mx.moonep_grad_table(none), 1.0, norm, work())
        assert norm.item() == 0


def test_many_tensors_same_bits_every_time(gpu_ready):
    g = gen(3)
    src = [torch.randn(1 + 37 * i % 900, generator=g, device="cuda") for i in range(3000)]
    table, norm = mx.moonep_grad_table(src), torch.empty(1, device="cuda")
    ss = [torch.empty(1, device="cuda", dtype=torch.float64) for _ in range(3)]
    for s in ss:
        mx.moonep_grad_norm(table, norm, work(), s)
    want = float((torch.cat(src).double() ** 2).sum())
    assert ss[0].item() == ss[1].item() == ss[2].item()
    assert abs(ss[0].item() - want) <= 1e-12 * want


def test_a_run_longer_than_the_usual(gpu_ready):
    a = torch.randn(100003, generator=gen(4), device="cuda")
    o = torch.empty_like(a)
    table = torch.tensor([[a.data_ptr(), o.data_ptr(), a.numel(), mx.F32]], device="cuda")
    norm = torch.empty(1, device="cuda")
    mx.moonep_grad_clip(table, 1e9, norm, work())
    assert torch.equal(o, a)
    assert abs(norm.item() - a.double().norm().item()) <= 2.0 ** -23 * norm.item()


def test_graph_and_stream(gpu_ready):
    g = gen(5)
    a, b = torch.randn(5000, generator=g, device="cuda"), torch.randn(77, generator=g, device="cuda").bfloat16()
    oa, ob = torch.empty_like(a), torch.empty_like(b)
    table, norm, ws = mx.moonep_grad_table([a, b], [oa, ob]), torch.empty(1, device="cuda"), work()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        mx.moonep_grad_clip(table, 1.0, norm, ws)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.moonep_grad_clip(table, 1.0, norm, ws)
    for k in range(3):
        a.normal_()
        graph.replay()
        total = math.sqrt(float((a.double() ** 2).sum() + (b.double() ** 2).sum()))
        assert abs(norm.item() - total) <= 2.0 ** -23 * total
        assert ((oa.double() - a.double() / total).abs() <= 2.0 ** -22 * a.double().abs()).all()
