"""A training step through the C-ABI: a shared projection with low-rank adapters, the experts behind a plan with
replicas, their backward, the replicas' reduction, and the clipping of all gradients.  Inputs are small integers,
sparse enough that every value is exact in bf16 and every sum in fp32, so that fp64 autograd over the layer's
definition has to be met to the bit, whatever the order of sums."""
import math

import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, R=4, E=8, S=40, K=2, D=64, H=128, F=128, M=3, rank=16, B=1, seed=0):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.s, self.sa = mx.Shape(R, E, S, K, H), mx.Shape(1, M + 1, R * S, 1, 8)
        self.dims = R, E, S, K, D, H, F, M, rank, B
        N = self.N = R * S
        dev = "cuda"

        def ints(*shape, keep):
            v = torch.randint(0, 2, shape, generator=g, device=dev) * 2 - 1
            return (v * (torch.rand(shape, generator=g, device=dev) < keep)).bfloat16()

        self.z, self.dy = ints(N, D, keep=0.15), ints(N, H, keep=0.1)
        self.Ws = ints(H, D, keep=0.1)
        self.w = torch.cat([ints(E, F * H, keep=0.03), ints(E, H * F, keep=0.03)], 1)  # rows of both matrices
        self.ad = mx.Adapters(M, rank, D, H)
        self.bank = torch.cat([ints(M, rank * D, keep=0.1), ints(M, H * rank, keep=0.05)], 1)
        self.scale = torch.tensor([1.0, 2.0, 0.5][:M], device=dev)
        ids = torch.randint(0, M + 1, (N,), generator=g, device=dev)
        self.ids = ids.int()
        logits = torch.randn((N, E), generator=g, device=dev) + 1.5 * torch.randn(E, generator=g, device=dev)
        self.topk = torch.topk(logits, K, dim=1).indices.int().contiguous().view(-1)
        self.gates = torch.tensor([0.5, 0.25], device=dev).repeat(N)
        bf = lambda *n: torch.full(n, float("nan"), dtype=torch.bfloat16, device=dev)  # noqa: E731
        f32 = lambda *n: torch.full(n, float("nan"), device=dev)  # noqa: E731
        NK = N * K
        self.b, self.ba = mx.allocate(self.s), mx.allocate(self.sa)
        self.wslot = torch.empty(E + R, dtype=torch.int32, device=dev)
        self.pool = torch.zeros((R * B, 2 * F * H), dtype=torch.bfloat16, device=dev)
        self.base, self.x, self.u, self.h, self.o, self.y = bf(N, H), bf(N, H), f32(N, rank), bf(NK, F), bf(NK, H), bf(N, H)
        self.d_o, self.d_g, self.d_h, self.d_buf = bf(NK, H), f32(NK), bf(NK, F), bf(NK, H)
        self.d_x, self.d_base, self.d_z = bf(N, H), bf(N, D), bf(N, D)
        self.d_bank, self.home = f32(M, self.bank.shape[1]), f32(E, 2 * F * H)
        self.rep = torch.zeros((E + R, 2 * F * H), device=dev)
        self.ws = torch.empty(mx.moonep_adapter_workspace_bytes(self.sa, self.ad), dtype=torch.uint8, device=dev)
        self.wsb = torch.empty(mx.moonep_adapter_bwd_workspace_bytes(self.sa, self.ad), dtype=torch.uint8, device=dev)
        self.wsg = torch.empty(mx.GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
        self.clipped = [f32(*t.shape) for t in (self.home, self.d_bank)]
        self.norm = f32(1)
        self.table = mx.moonep_grad_table([self.home, self.d_bank], self.clipped)

    def run(self, accumulate=False, max_norm=1.0):
        R, E, S, K, D, H, F, M, rank, B = self.dims
        s, b, n = self.s, self.b, F * H
        mx.plan_step(self.ba, self.ids)
        mx.plan_step(b, self.topk)
        mx.moonep_weight_slots(s, b.plan, B, self.wslot)
        mx.moonep_prefetch_weights(s, b.plan, self.wslot, B, 4 * n, self.w, self.pool)
        # forward
        self.base.copy_(self.z.float() @ self.Ws.float().T)
        mx.moonep_adapter(self.sa, self.ad, self.ids, self.ba.src_of_slot, self.z, self.bank, self.scale, self.base, self.u,
                          self.x, self.ws)
        mx.moonep_dispatch(s, self.x, b.slot_of, b.buf)
        mx.moonep_expert_gemm(s, b.plan, self.wslot, B, H, F, b.buf, self.w, self.pool, 2 * n, 0, self.h)
        self.h.clamp_(min=0)
        mx.moonep_expert_gemm(s, b.plan, self.wslot, B, F, H, self.h, self.w, self.pool, 2 * n, n, self.o)
        mx.moonep_combine(s, self.o, self.gates, b.slot_of, self.y)
        # backward
        mx.moonep_combine_bwd(s, self.dy, self.o, self.gates, b.slot_of, self.d_o, self.d_g)
        mx.moonep_expert_gemm_dx(s, b.plan, self.wslot, B, F, H, self.d_o, self.w, self.pool, 2 * n, n, self.d_h)
        mx.moonep_expert_gemm_dw(s, b.plan, F, H, self.h, self.d_o, accumulate, 2 * n, n, self.home, self.rep)
        self.d_h.mul_(self.h > 0)
        mx.moonep_expert_gemm_dx(s, b.plan, self.wslot, B, H, F, self.d_h, self.w, self.pool, 2 * n, 0, self.d_buf)
        mx.moonep_expert_gemm_dw(s, b.plan, H, F, b.buf, self.d_h, accumulate, 2 * n, 0, self.home, self.rep)
        mx.moonep_dispatch_bwd(s, self.d_buf, b.slot_of, self.d_x)
        self.d_base.copy_(self.d_x.float() @ self.Ws.float())
        mx.moonep_adapter_bwd(self.sa, self.ad, self.ids, self.ba.src_of_slot, self.ba.plan, self.z, self.u, self.d_x, self.bank,
                              self.scale, self.d_base, self.d_z, accumulate, self.d_bank, self.wsb)
        mx.moonep_replica_grad_reduce(s, b.plan, 2 * n, self.home, self.rep)
        mx.moonep_grad_clip(self.table, max_norm, self.norm, self.wsg)

    def reference(self):
        """y, and the gradients of <dy, y> with respect to z, the experts' matrices and the bank."""
        R, E, S, K, D, H, F, M, rank, B = self.dims
        leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
        z, w, bank = leaf(self.z), leaf(self.w), leaf(self.bank)
        A, Bm = bank[:, :rank * D].view(M, rank, D), bank[:, rank * D:].view(M, H, rank)
        x = z @ self.Ws.double().T
        for m in range(M):
            on = (self.ids == m).double()[:, None]
            x = x + on * self.scale[m].double() * (z @ A[m].T @ Bm[m].T)
        y = torch.zeros_like(x)
        for k in range(K):
            of = self.topk.view(-1, K)[:, k]
            for e in range(E):
                on = (of == e).double()[:, None]
                h = torch.relu(x @ w[e, :F * H].view(F, H).T)
                y = y + on * self.gates.view(-1, K)[:, k:k + 1].double() * (h @ w[e, F * H:].view(H, F).T)
        grads = torch.autograd.grad((y * self.dy.double()).sum(), (z, w, bank))
        return (y, *grads)

    def check(self, times=1, max_norm=1.0):
        y, d_z, d_w, d_bank = self.reference()
        # bf16's 8 bits hold multiples of 1/2 up to 128 (scales of 1/2 at least) and of 1/4 up to 64 (gates)
        for t in (self.x, self.h, self.o):
            assert t.abs().max() <= 128
        for t in (self.d_h, self.d_buf, self.d_x):
            assert t.abs().max() <= 64
        assert torch.equal(self.y.double(), y) and torch.equal(self.d_z.double(), d_z)
        assert torch.equal(self.home.double(), times * d_w) and torch.equal(self.d_bank.double(), times * d_bank)
        assert (self.rep == 0).all()
        total = times * math.sqrt(float((d_w ** 2).sum() + (d_bank ** 2).sum()))
        assert abs(self.norm.item() - total) <= 2.0 ** -23 * total
        for c, g in zip(self.clipped, (times * d_w, times * d_bank)):
            assert ((c.double() - g * min(1.0, max_norm / total)).abs() <= 2.0 ** -22 * g.abs()).all()


def test_step(gpu_ready):
    t = Step()
    t.run()
    assert t.b.plan_fields()["n_rep"] > 0
    t.check()
    t.run(accumulate=True, max_norm=1e9)  # a second microbatch on top
    t.check(times=2, max_norm=1e9)


@pytest.mark.parametrize("shape", [dict(R=1, E=4, S=300, D=128, F=256), dict(R=2, E=16, S=7, rank=8, B=4),
                                   dict(R=4, E=8, S=600, D=192, B=0)])
def test_other_shapes(gpu_ready, shape):
    t = Step(seed=1, **shape)
    t.run()
    t.check()


def test_captured_step(gpu_ready):
    """The whole step as a graph, replayed over new inputs, with eager work in between; two such graphs share
    nothing, and their replays interleave."""
    steps = [Step(seed=2), Step(seed=3, S=90)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in steps:
            t.run()
    side.synchronize()
    graphs = []
    for t in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t.run()
        graphs.append(graph)
    for k in range(3):
        for t in steps:
            t.dy.copy_(t.dy[torch.randperm(t.N, generator=t.g, device="cuda")])
            t.ids.copy_(t.ids.roll(k + 1))
            t.topk.copy_(t.topk.roll(2))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for t in steps:
            t.check()
        if k == 1:  # eager in between, on the same buffers
            for t in steps:
                t.run()
                t.check()


def test_two_steps_on_two_streams(gpu_ready):
    steps = [Step(seed=4, S=200), Step(seed=5, S=60, E=16)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for st, t in zip(streams, steps):
        with torch.cuda.stream(st):
            t.run()
    torch.cuda.synchronize()
    for t in steps:
        t.check()
