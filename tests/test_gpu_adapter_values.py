"""Adapters on an MI355X with the values at which split products can go wrong: infinities
and NaN in matrices and rows, sums at the end of fp32's range, and gradients that need all
24 bits of u and du."""
import pytest
import torch

from test_gpu_adapters import Case

pytestmark = pytest.mark.gpu

INF = float("inf")


def same_kind_and_near(got, want, tol):
    """NaN and the infinities where the fp64 formula has them, and within tol elsewhere."""
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isposinf(), want.isposinf()) and torch.equal(got.isneginf(), want.isneginf())
    fin = want.isfinite()
    assert ((got - want).abs()[fin] <= tol[fin]).all()


@pytest.mark.parametrize("order", [True, False])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 128])
@pytest.mark.parametrize("N", [40, 2200])
def test_infinities_in_the_forward(gpu_ready, N, rank, order):
    """An infinite weight gives its column infinities of u's signs, an infinite row its results."""
    c = Case(N, 4, rank, 64, 72, seed=11)
    A, B = c.mats(c.bank)
    B[1, 5, 3] = INF
    B[2, 70, rank - 1] = -INF
    B[3, 8, 1], B[3, 8, 2] = INF, -INF
    for m in (0, 1):
        c.x[torch.nonzero(c.ids == m)[0, 0], 9] = INF
    c.forward(order)
    for m in range(4):
        at, s = c.ids == m, c.scale[m].double()
        x, a, b, base = c.x[at].double(), A[m].double(), B[m].double(), c.base[at].double()
        u = x @ a.T
        same_kind_and_near(c.u[at], u, 64 * 2.0 ** -23 * (x.abs() @ a.abs().T))
        su = s * c.u[at].double()
        want, mag = base + su @ b.T, su.abs() @ b.abs().T
        # the split to 16 bits, the scale's rounding, 2 rank additions and that of base; bf16's rounding
        tol = 1.01 * (2.0 ** -16 + (2 * rank + 2) * 2.0 ** -23) * mag + 2.0 ** -23 * (base.abs() + mag)
        same_kind_and_near(c.y[at], want, tol + 2.0 ** -8 * want.abs())


def all_gradients(c):
    d_x = torch.full_like(c.dx_base, 7.0)
    d_bank = torch.full((c.M, c.ad.stride), 7.0, device="cuda")
    c.backward(d_bank=d_bank, d_x=d_x, dx_base=c.dx_base)
    return d_x, d_bank


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 128])
@pytest.mark.parametrize("N", [60, 1000, 2200, 9000])
def test_infinities_in_the_backward(gpu_ready, N, rank):
    """Infinite weights, rows and gradients, and a NaN, each of another adapter or place."""
    c = Case(N, 5, rank, 64, 72, seed=12)
    c.u = torch.randn((N, rank), generator=c.g, device="cuda")
    A, B = c.mats(c.bank)
    A[1, 2, 6], A[1, 4, 60] = INF, -INF
    B[2, 9, 3] = INF
    first = lambda m, k=0: torch.nonzero(c.ids == m)[k, 0]  # noqa: E731
    c.x[first(3), 4], c.x[first(3, 1), 50] = INF, -INF
    c.x[first(3, 1), 4] = INF
    c.d_y[first(0), 8] = -INF
    c.x[first(4), 33] = float("nan")
    c.u[first(4), 5] = INF
    d_x, d_bank = all_gradients(c)
    dx, t_x, grads, tols = c.reference_backward()
    same_kind_and_near(d_x, dx, t_x)
    for got, want, tol in zip(c.mats(d_bank), grads, tols):
        same_kind_and_near(got, want, tol)


NEAR_THE_END = 255 * 2.0 ** 120 + 0.75 * 2.0 ** 120  # of fp32; its nearest bf16 is an infinity


@pytest.mark.parametrize("rank", [8, 24, 64, 128])
@pytest.mark.parametrize("N", [40, 2200])
def test_sums_at_the_end_of_fp32(gpu_ready, N, rank):
    """u and du that fp32 holds and bf16 does not: finite results where the formula's are."""
    c = Case(N, 3, rank, 64, 72, seed=13)
    A, B = c.mats(c.bank)
    c.scale.fill_(1.0)
    sign = torch.where(torch.rand(N, generator=c.g, device="cuda") < 0.5, -1.0, 1.0)
    tiny = 2.0 ** -100
    c.x.zero_()
    c.x[:, 0], c.x[:, 1] = 255 * 2.0 ** 120 * sign, 0.75 * 2.0 ** 120 * sign
    A.fill_(1.0)
    B *= tiny
    c.base *= tiny
    c.forward()
    assert (c.u[c.ids < 3].abs() == NEAR_THE_END).all()
    c.check_forward()
    # d_y tiny: dB takes u
    c.d_y *= tiny
    c.dx_base *= tiny
    B /= tiny
    A.copy_(torch.randn(A.shape, generator=c.g, device="cuda"))
    c.x.copy_(torch.randn(c.x.shape, generator=c.g, device="cuda"))
    c.check_backward(*all_gradients(c))
    # du as large: d_x and dA take it
    c.u *= tiny * tiny
    c.d_y.zero_()
    c.d_y[:, 0], c.d_y[:, 1] = 255 * 2.0 ** 120 * sign, 0.75 * 2.0 ** 120 * sign
    B.fill_(1.0)
    A *= tiny
    c.x *= tiny
    c.check_backward(*all_gradients(c))


EXACT = [
    # N, M, rank: few rows in one piece and several, many rows, adapters over several chunks
    (40, 5, 8), (40, 40, 24), (700, 9, 72), (200, 3, 128), (2200, 6, 8), (2200, 90, 40),
    (9000, 1, 24), (9000, 2, 72), (9000, 3, 128), (5000, 3, 64), (5000, 2, 16), (33000, 2, 32),
]


def one_row_each(c, n):
    """For every adapter with rows, one of them for each of n columns."""
    rows = [torch.nonzero(c.ids == m)[:, 0] for m in range(c.M)]
    return [r[torch.randint(0, r.numel(), (n,), generator=c.g, device="cuda")] if r.numel() else None for r in rows]


@pytest.mark.parametrize("N,M,rank", EXACT)
def test_all_bits_of_u_reach_the_gradient(gpu_ready, N, M, rank):
    """d_y is 1 in one row of each column and 0 elsewhere: dB holds rows of u, to the bit."""
    c = Case(N, M, rank, 64, 72, seed=14)
    c.scale.fill_(1.0)
    c.u = torch.randn((N, rank), generator=c.g, device="cuda")
    c.d_y.zero_()
    hot, cols = one_row_each(c, c.out), torch.arange(c.out, device="cuda")
    for r in hot:
        if r is not None:
            c.d_y[r, cols] = 1.0
    d_bank = torch.full((M, c.ad.stride), 7.0, device="cuda")
    c.backward(d_bank=d_bank)
    dB = c.mats(d_bank)[1]
    for m, r in enumerate(hot):
        assert torch.equal(dB[m], c.u[r] if r is not None else torch.zeros_like(dB[m])), m


@pytest.mark.parametrize("N,M,rank", EXACT)
def test_all_bits_of_du_reach_the_gradient(gpu_ready, N, M, rank):
    """du is an integer of 24 bits, in exact sums of three products; x is 1 in one row of
    each column and 0 elsewhere: dA holds rows of du, to the bit."""
    c = Case(N, M, rank, 64, 72, seed=15)
    c.scale.fill_(1.0)
    c.d_y.zero_()
    c.d_y[:, :3] = torch.where(torch.rand((N, 3), generator=c.g, device="cuda") < 0.5, -1.0, 1.0).bfloat16()
    _, B = c.mats(c.bank)
    digits = torch.randint(128, 256, (M, 3, rank), generator=c.g, device="cuda").float()
    B[:, :3] = (digits * torch.tensor([65536.0, 256.0, 1.0], device="cuda")[None, :, None]).bfloat16()
    c.x.zero_()
    hot, cols = one_row_each(c, c.inp), torch.arange(c.inp, device="cuda")
    for r in hot:
        if r is not None:
            c.x[r, cols] = 1.0
    c.u.zero_()
    d_bank = torch.full((M, c.ad.stride), 7.0, device="cuda")
    c.backward(d_bank=d_bank)
    dA, dB = c.mats(d_bank)
    assert (dB == 0).all()
    for m, r in enumerate(hot):
        du = c.d_y[r, :3].double() @ B[m, :3].double() if r is not None else torch.zeros((c.inp, rank), device="cuda")
        assert torch.equal(dA[m], du.T.float()), m


WIDE = [
    # more rows than few, of contractions in several parts, at the ranks above 32
    (1100, 5, 64, 2048, 2056), (1100, 4, 40, 2056, 4096), (1100, 3, 128, 4096, 2048), (1100, 3, 96, 2048, 4104),
    # rows and results past the caches (over 128 MiB) at every form of the rank
    (9000, 5, 24, 8192, 8192), (9000, 4, 64, 8200, 8192), (9000, 3, 128, 8192, 8200),
]


@pytest.mark.parametrize("case", WIDE)
def test_wide_rows(gpu_ready, case):
    c = Case(*case, gap=8, seed=16)
    c.forward()
    c.check_forward()
    d_x, d_bank = all_gradients(c)
    c.check_backward(d_x, d_bank)
    for m in c.mats(d_bank):
        m.fill_(7.0)
    assert (d_bank == 7.0).all()
