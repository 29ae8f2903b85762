"""The router captured into a graph and replayed, with the program's own work between the replays: forward and
backward, bf16 and fp32 logits, with the loss and without; and the backward captured while an eager one has just
run on the same tensors."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx
from gpu_harness import to_dev
from test_gpu_router import SIG, SOFT

pytestmark = pytest.mark.gpu


class Router:
    def __init__(self, shape, opts, loss):
        dev, s = "cuda", shape
        t = torch.bfloat16 if opts.logits_type == mx.BF16 else torch.float32
        self.s, self.o, self.with_loss = s, opts, loss
        self.logits, self.d_logits = torch.empty((s.N, s.E), dtype=t, device=dev), torch.empty((s.N, s.E), dtype=t, device=dev)
        self.ids, self.gates = torch.empty(s.NK, dtype=torch.int32, device=dev), torch.empty(s.NK, device=dev)
        self.d_gates, self.d_loss = torch.empty(s.NK, device=dev), torch.empty(1, device=dev)
        if loss:
            self.counts = torch.empty((opts.groups, s.E), dtype=torch.int32, device=dev)
            self.prob, self.loss = torch.empty((opts.groups, s.E), device=dev), torch.empty(1, device=dev)
            self.ws = torch.empty(mx.moonep_router_workspace_bytes(s, opts), dtype=torch.uint8, device=dev)

    def load(self, seed):
        rng = np.random.default_rng(seed)
        self.logits.copy_(to_dev(rng.standard_normal((self.s.N, self.s.E)).astype(np.float32)))
        self.d_gates.copy_(to_dev(rng.standard_normal(self.s.NK).astype(np.float32)))
        self.d_loss.fill_(0.1 + seed)
        for t in self.outputs().values():
            t.view(torch.uint8).fill_(0x5B)
        if self.with_loss:
            self.ws.fill_(0xEE)

    def step(self):
        if self.with_loss:
            mx.moonep_router(self.s, self.o, self.logits, self.ids, self.gates, self.counts, self.prob, self.loss, self.ws)
        else:
            mx.moonep_router(self.s, self.o, self.logits, self.ids, self.gates)
        mx.moonep_router_bwd(self.s, self.o, self.logits, self.ids, self.counts if self.with_loss else None,
                             self.d_gates, self.d_loss if self.with_loss else None, self.d_logits)

    def outputs(self):
        out = dict(ids=self.ids, gates=self.gates, d_logits=self.d_logits)
        if self.with_loss:
            out.update(counts=self.counts, prob=self.prob, loss=self.loss)
        return out

    def snapshot(self):
        return {k: v.view(torch.uint8).cpu().numpy().copy() for k, v in self.outputs().items()}


@pytest.mark.parametrize("loss", [False, True], ids=["no_loss", "loss"])
@pytest.mark.parametrize("E,K,score,normalize,bf16", [(64, 8, SOFT, False, True), (130, 1, SIG, True, True),
                                                      (256, 8, SIG, True, False), (40, 20, SOFT, True, False)])
def test_captured_and_replayed(E, K, score, normalize, bf16, loss):
    print(f"[case] graph of the router E={E} K={K} score={score} norm={normalize} bf16={bf16} loss={loss}", flush=True)
    r = Router(mx.Shape(1, E, 618, K, 16), mx.RouterOpts(score, normalize, 2, int(bf16), 1.5), loss)
    want = {}
    for seed in range(3):
        r.load(seed)
        r.step()
        torch.cuda.synchronize()
        want[seed] = r.snapshot()
    assert not np.array_equal(want[0]["ids"], want[1]["ids"])
    r.load(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.step()
    for i in range(6):
        r.load(i % 3)
        noise = torch.randn(256, 256, device="cuda") @ torch.randn(256, 256, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in r.snapshot().items():
            np.testing.assert_array_equal(v, want[i % 3][k], err_msg=f"replay {i}: {k}")
        del noise
        r.load(i % 3)
        r.step()  # eager, between the replays
        torch.cuda.synchronize()
        for k, v in r.snapshot().items():
            np.testing.assert_array_equal(v, want[i % 3][k], err_msg=f"eager after replay {i}: {k}")
