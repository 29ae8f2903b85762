"""The backward of the experts' products on an MI355X: d_x and the weight
gradients against fp64 sums over the plan's segments, bit for bit where every
sum is exact, and against differences of the forward product."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx
import synth

pytestmark = pytest.mark.gpu


def setup(R, E, S, K, seed=0, skew=1.0):
    """A layer planned on the device, and its segments (row0, rows, expert, replica or -1)."""
    s = mx.Shape(R, E, S, K, 64)
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((s.N, E), generator=g, device="cuda") + skew * torch.randn(E, generator=g, device="cuda")
    topk = torch.topk(logits, K, dim=1).indices.int().contiguous().view(-1)
    b = mx.allocate(s)
    mx.plan_step(b, topk)
    f = b.plan_fields()
    L = E // R
    segs = [((e // L) * s.C + int(f["home_row_off"][e]), int(f["keep"][e]), e, -1) for e in range(E)]
    segs += [(int(f["rep_host"][j]) * s.C + int(f["rep_row_off"][j]), int(f["rep_count"][j]),
              int(f["rep_expert"][j]), j) for j in range(f["n_rep"])]
    return s, b, segs, g


def values(shape, g, integers, std=1.0):
    if integers:  # products and sums of these are exact in fp32 (below 2^24) in any order
        return torch.randint(-3, 4, shape, generator=g, device="cuda").bfloat16()
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * std


CASES = [
    # R, E, S, K, in, out, B: segments below, at and above a tile; edges of column blocks
    (1, 1, 1, 1, 64, 128, 0),
    (1, 4, 300, 1, 64, 128, 0),
    (2, 4, 77, 2, 320, 384, 1),
    (4, 16, 37, 2, 192, 256, 0),
    (4, 8, 513, 3, 576, 128, 2),
    (8, 32, 130, 4, 256, 640, 4),
    (2, 64, 9, 4, 1088, 256, 3),
    # enough rows, and enough items, for the large tiles
    (4, 4, 16384, 1, 320, 128, 1),
    (8, 16, 4099, 2, 576, 128, 1),
    (4, 64, 40, 2, 832, 384, 0),
    (2, 32, 300, 4, 1088, 640, 1),
    # d_x: small tiles of 128 rows, each on a CU and not, and of 64 rows in several rounds
    (2, 4, 1000, 2, 640, 256, 1),
    (8, 16, 1500, 2, 576, 128, 1),
    (8, 64, 500, 4, 704, 128, 2),
    (4, 64, 200, 4, 1344, 128, 2),
]


def weights_of(segs, wslot, w_home, pool, n_slots):
    ws = wslot.tolist()
    for row0, n, e, j in segs:
        pooled = j >= 0 and 0 <= ws[j] < n_slots
        yield row0, n, (pool[ws[j]] if pooled else w_home[e])


@pytest.mark.parametrize("integers", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_dx(gpu_ready, case, integers):
    R, E, S, K, kin, kout, B = case
    s, b, segs, g = setup(R, E, S, K)
    stride, at = kin * kout + 24, 16
    w = torch.full((E, stride), float("nan"), device="cuda").bfloat16()
    w[:, at:at + kin * kout] = values((E, kin * kout), g, integers, kin ** -0.5)
    wslot = torch.empty(E + R, dtype=torch.int32, device="cuda")
    mx.moonep_weight_slots(s, b.plan, B, wslot)
    pool = torch.zeros((R * B, stride), dtype=torch.bfloat16, device="cuda")
    mx.moonep_prefetch_weights(s, b.plan, wslot, B, stride * 2, w, pool)
    dy = values((s.NK, kout), g, integers)
    dx = torch.full((s.NK, kin), float("nan"), device="cuda").bfloat16()
    mx.moonep_expert_gemm_dx(s, b.plan, wslot, B, kin, kout, dy, w, pool, stride, at, dx)
    for row0, n, wr in weights_of(segs, wslot, w, pool, R * B):
        if not n:
            continue
        d, m = dy[row0:row0 + n].double(), wr[at:at + kin * kout].double().view(kout, kin)
        want, got = d @ m, dx[row0:row0 + n]
        if integers:
            assert torch.equal(got, want.bfloat16())
        else:
            # one rounding to bf16; kout additions in fp32, each within 2^-23
            tol = 2.0 ** -8 * want.abs() + kout * 2.0 ** -23 * (1 + 2.0 ** -8) * (d.abs() @ m.abs())
            assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("integers", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_dw(gpu_ready, case, integers, accumulate):
    R, E, S, K, kin, kout, _ = case
    s, b, segs, g = setup(R, E, S, K)
    G, at = kin * kout + 7, 5
    x, dy = values((s.NK, kin), g, integers), values((s.NK, kout), g, integers)
    home = torch.randint(-9, 10, (E, G), generator=g, device="cuda").float()
    rep = torch.randint(-9, 10, (E + R, G), generator=g, device="cuda").float()
    home0, rep0 = home.clone(), rep.clone()
    mx.moonep_expert_gemm_dw(s, b.plan, kin, kout, x, dy, accumulate, G, at, home, rep)
    want_home, want_rep = home0.double(), rep0.double()
    tol_home, tol_rep = torch.zeros_like(want_home), torch.zeros_like(want_rep)
    for row0, n, e, j in segs:
        d, v = dy[row0:row0 + n].double(), x[row0:row0 + n].double()
        out, tol = (want_home[e], tol_home[e]) if j < 0 else (want_rep[j], tol_rep[j])
        old = out[at:at + kin * kout].clone() if accumulate else 0.0
        out[at:at + kin * kout] = old + (d.T @ v).view(-1)
        # n additions in fp32, each within 2^-23, and one of the old value
        tol[at:at + kin * kout] = (n + 1) * 2.0 ** -23 * ((d.abs().T @ v.abs()).view(-1) + 9)
    if integers:
        assert torch.equal(home.double(), want_home) and torch.equal(rep.double(), want_rep)
    else:
        assert ((home.double() - want_home).abs() <= tol_home).all()
        assert ((rep.double() - want_rep).abs() <= tol_rep).all()


def test_gradients_are_the_forwards_differences(gpu_ready):
    """y is linear in x and in W: with small integers every sum is exact, so the
    gradient of <d_y, y> is the forward's difference, to the last bit."""
    R, E, S, K, kin, kout, B = 2, 8, 21, 2, 128, 128, 4
    s, b, segs, g = setup(R, E, S, K)
    small = lambda shape: torch.randint(-1, 2, shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, dy, w = small((s.NK, kin)), small((s.NK, kout)), small((E, kin * kout))
    wslot = torch.full((E + R,), -1, dtype=torch.int32, device="cuda")
    pool = torch.zeros((R * B, kin * kout), dtype=torch.bfloat16, device="cuda")

    def forward(x, w):
        y = torch.empty((s.NK, kout), dtype=torch.bfloat16, device="cuda")
        mx.moonep_expert_gemm(s, b.plan, wslot, B, kin, kout, x, w, pool, kin * kout, 0, y)
        assert y.abs().max() <= 256  # exact in bf16
        return y.double()

    dx = torch.empty((s.NK, kin), dtype=torch.bfloat16, device="cuda")
    mx.moonep_expert_gemm_dx(s, b.plan, wslot, B, kin, kout, dy, w, pool, kin * kout, 0, dx)
    home = torch.zeros((E, kin * kout), device="cuda")
    rep = torch.zeros((E + R, kin * kout), device="cuda")
    mx.moonep_expert_gemm_dw(s, b.plan, kin, kout, x, dy, False, kin * kout, 0, home, rep)
    mx.moonep_replica_grad_reduce(s, b.plan, kin * kout, home, rep)
    y0 = (dy.double() * forward(x, w)).sum()
    ex, ew = small(x.shape), small(w.shape)
    assert (dy.double() * forward(x + ex, w)).sum() - y0 == (dx.double() * ex.double()).sum()
    assert (dy.double() * forward(x, w + ew)).sum() - y0 == (home.double() * ew.double()).sum()


def test_what_stands_behind_a_segment_is_not_summed(gpu_ready):
    """Rows of other segments around a short one hold NaN: it is not touched by them."""
    s, b, segs, g = setup(1, 8, 40, 1)
    kin, kout = 128, 128
    row0, n, e, _ = max((q for q in segs if q[1] % 64), key=lambda q: q[1])
    x = torch.full((s.NK, kin), float("nan"), device="cuda").bfloat16()
    dy = torch.full((s.NK, kout), float("inf"), device="cuda").bfloat16()
    x[row0:row0 + n], dy[row0:row0 + n] = values((n, kin), g, True), values((n, kout), g, True)
    home = torch.empty((8, kin * kout), device="cuda")
    rep = torch.empty((9, kin * kout), device="cuda")
    mx.moonep_expert_gemm_dw(s, b.plan, kin, kout, x, dy, False, kin * kout, 0, home, rep)
    want = dy[row0:row0 + n].double().T @ x[row0:row0 + n].double()
    assert torch.equal(home[e].double().view(kout, kin), want)


def test_no_rows(gpu_ready):
    s = mx.Shape(2, 4, 0, 2, 64)
    b = mx.allocate(s)
    mx.plan_step(b, torch.empty(0, dtype=torch.int32, device="cuda"))
    home, rep = torch.ones((4, 64 * 128), device="cuda"), torch.ones((6, 64 * 128), device="cuda")
    none = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    mx.moonep_expert_gemm_dw(s, b.plan, 64, 128, none, none, True, 64 * 128, 0, home, rep)
    assert (home == 1).all() and (rep == 1).all()
    mx.moonep_expert_gemm_dw(s, b.plan, 64, 128, none, none, False, 64 * 128, 0, home, rep)
    assert (home == 0).all() and (rep == 1).all()


@pytest.mark.parametrize("level", [0.0, 4.0])
def test_sweep_rows(gpu_ready, level):
    """Segments of the benchmark's routing, balanced and skewed, on a narrow layer."""
    w = synth.sweep_workload(level, seed=0)
    topk, _ = synth.routing(w, 0)
    s = mx.Shape(w.R, w.E, w.S, w.K, 64)
    b = mx.allocate(s)
    mx.plan_step(b, torch.from_numpy(np.ascontiguousarray(topk)).to("cuda"))
    f = b.plan_fields()
    g = torch.Generator(device="cuda").manual_seed(1)
    kin, kout = 64, 128
    x, dy = values((s.NK, kin), g, True), values((s.NK, kout), g, True)
    home = torch.empty((w.E, kin * kout), device="cuda")
    rep = torch.zeros((w.E + w.R, kin * kout), device="cuda")
    mx.moonep_expert_gemm_dw(s, b.plan, kin, kout, x, dy, False, kin * kout, 0, home, rep)
    mx.moonep_replica_grad_reduce(s, b.plan, kin * kout, home, rep)
    expert = torch.from_numpy(np.ascontiguousarray(topk)).to("cuda").long()[b.src_of_slot.long()]
    for e in range(0, w.E, 7):
        rows = expert == e
        assert torch.equal(home[e].double().view(kout, kin), dy[rows].double().T @ x[rows].double())
    assert f["n_rep"] > 0 or level == 0.0
