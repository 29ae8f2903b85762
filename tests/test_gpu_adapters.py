"""Low-rank adapters on an MI355X: forward and backward against fp64 formulas,
and against differences of the forward where every sum is exact."""
import pytest
import torch

import load_balancing_amd as mx

pytestmark = pytest.mark.gpu

NAN = float("nan")


class Case:
    """N rows, M adapters (ids M: none), planned by the framework's own plan."""

    def __init__(self, N, M, rank, inp, out, none=0.2, seed=0, integers=False, gap=0, runs=None):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.N, self.M, self.rank, self.inp, self.out = N, M, rank, inp, out
        self.s = mx.Shape(1, M + 1, N, 1, 8)
        stride = rank * (inp + out) + 3 * gap
        self.ad = mx.Adapters(M, rank, inp, out, stride, gap, 2 * gap + rank * inp)
        ids = torch.randint(0, M, (N,), generator=g, device="cuda")
        if runs:  # whole sequences after one another
            ids = ids[torch.arange(N, device="cuda") // runs]
        ids[torch.rand(N, generator=g, device="cuda") < none] = M
        self.ids = ids.int()
        self.b = mx.allocate(self.s)
        mx.plan_step(self.b, self.ids)
        self.order, self.plan = self.b.src_of_slot, self.b.plan
        if integers:
            v = lambda *shape: torch.randint(-1, 2, shape, generator=g, device="cuda").bfloat16()  # noqa: E731
            self.scale = torch.full((M,), 2.0, device="cuda")
        else:
            v = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
            self.scale = 0.5 + torch.rand(M, generator=g, device="cuda")
        self.x, self.base, self.d_y, self.dx_base = v(N, inp), v(N, out), v(N, out), v(N, inp)
        self.bank = torch.full((M, stride), NAN, device="cuda").bfloat16()
        A, B = self.mats(self.bank)
        A[:], B[:] = v(M, rank, inp), v(M, out, rank)
        if not integers:
            A *= inp ** -0.5
            B *= 0.3 * rank ** -0.5
        self.y = torch.full((N, out), NAN, device="cuda").bfloat16()
        self.u = torch.full((N, rank), NAN, device="cuda")

    def mats(self, bank):
        a, r = self.ad, self.rank
        return (bank[:, a.a_offset:a.a_offset + r * self.inp].unflatten(1, (r, self.inp)),
                bank[:, a.b_offset:a.b_offset + r * self.out].unflatten(1, (self.out, r)))

    def work(self, bwd=False):
        n = (mx.moonep_adapter_bwd_workspace_bytes if bwd else mx.moonep_adapter_workspace_bytes)(self.s, self.ad)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in fp32

    def forward(self, order=True, **k):
        mx.moonep_adapter(self.s, self.ad, self.ids, self.order if order else None, self.x, self.bank, self.scale,
                          k.get("base", self.base), self.u, k.get("y", self.y), k.get("ws", self.work()))

    def backward(self, accumulate=False, d_bank=None, d_x=None, dx_base=None, ws=None):
        mx.moonep_adapter_bwd(self.s, self.ad, self.ids, self.order, self.plan, self.x, self.u, self.d_y, self.bank,
                              self.scale, dx_base, d_x, accumulate, d_bank, self.work(True) if ws is None else ws)

    def check_forward(self):
        A, B = (m.double() for m in self.mats(self.bank))
        x, base = self.x.double(), self.base.double()
        for m in range(self.M + 1):
            at = self.ids == m
            if m == self.M:
                assert (self.u[at] == 0).all() and torch.equal(self.y[at], self.base[at])
                continue
            u, e_u = x[at] @ A[m].T, self.inp * 2.0 ** -23 * (x[at].abs() @ A[m].abs().T)
            assert ((self.u[at].double() - u).abs() <= e_u).all()
            s = self.scale[m].double()
            su = s * u
            y = base[at] + su @ B[m].T
            mag = su.abs() @ B[m].abs().T
            # u's error through the product; the split to 16 bits, the scale's rounding, 2 rank
            # additions in fp32 and that of base; one rounding to bf16
            tol = s * (e_u @ B[m].abs().T) + (2.0 ** -16 + (2 * self.rank + 2) * 2.0 ** -23) * mag
            tol = 1.01 * tol + 2.0 ** -23 * (base[at].abs() + mag) + 2.0 ** -8 * y.abs()
            assert ((self.y[at].double() - y).abs() <= tol).all(), m

    def reference_backward(self):
        """d_x, d_bank windows (A, B), and tolerances of each."""
        A, B = (m.double() for m in self.mats(self.bank))
        x, u, dy = self.x.double(), self.u.double(), self.d_y.double()
        dx, t_x = self.dx_base.double(), torch.zeros_like(self.dx_base, dtype=torch.float64)
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
        tA, tB = torch.zeros_like(A), torch.zeros_like(B)
        e = 2.0 ** -23
        for m in range(self.M):
            at, s = self.ids == m, self.scale[m].double()
            n = int(at.sum())
            du = s * (dy[at] @ B[m])
            e_du = (self.out + 1) * e * s * (dy[at].abs() @ B[m].abs())
            add = du @ A[m]
            mag = du.abs() @ A[m].abs()
            t_x[at] = 1.01 * (e_du @ A[m].abs() + (2.0 ** -16 + (2 * self.rank + 2) * e) * mag
                              ) + e * (dx[at].abs() + mag)
            dx[at] += add
            t_x[at] += 2.0 ** -8 * dx[at].abs()
            dA[m], dB[m] = du.T @ x[at], s * (dy[at].T @ u[at])
            # three bf16 parts of every value: 3 n additions, and those that join 64 chunks
            tA[m] = 1.01 * (e_du.T @ x[at].abs() + (3 * n + 66) * e * (du.abs().T @ x[at].abs()))
            tB[m] = 1.01 * (3 * n + 67) * e * s * (dy[at].abs().T @ u[at].abs())
        return dx, t_x, (dA, dB), (tA, tB)

    def check_backward(self, d_x, d_bank, old=None):
        dx, t_x, grads, tols = self.reference_backward()
        if d_x is not None:
            assert ((d_x.double() - dx).abs() <= t_x).all()
            none = self.ids == self.M
            assert torch.equal(d_x[none], self.dx_base[none])
        if d_bank is not None:
            for got, want, tol, was in zip(self.mats(d_bank), grads, tols, self.mats(old) if old is not None else (0, 0)):
                if old is not None:
                    was = was.double()
                    tol = tol + 2.0 ** -23 * (was.abs() + want.abs())
                    want = want + was
                assert ((got.double() - want).abs() <= tol).all()


CASES = [
    # N, M, rank, in, out
    (1, 1, 8, 8, 8),
    (3, 2, 16, 64, 72),
    (16, 16, 16, 256, 320),
    (17, 5, 24, 136, 40),
    (64, 64, 8, 512, 512),
    (127, 3, 32, 72, 1032),
    (300, 7, 40, 264, 200),
    (129, 2, 64, 1024, 96),
    (515, 40, 72, 88, 168),
    (200, 3, 128, 392, 136),
    (2049, 3, 16, 128, 136),
    (2500, 30, 32, 72, 264),
    (4100, 1, 64, 200, 64),
    (2113, 6, 128, 104, 72),
    (3000, 9, 56, 64, 128),
    # either side of what a wave, a workgroup and a launch take at once
    (256, 40, 64, 264, 520),
    (257, 40, 16, 520, 264),
    (250, 4, 128, 136, 72),
    (1024, 12, 24, 2056, 328),
    (4097, 90, 8, 64, 1096),
    (16385, 7, 16, 72, 136),
    (16500, 3, 128, 64, 72),
    (32769, 5, 32, 136, 64),
    (33000, 2, 64, 64, 200),
    (32770, 3, 96, 72, 64),
    (8192, 6, 16, 1024, 72),
    (8193, 6, 16, 1016, 72),
    (4097, 5, 32, 2048, 64),
    (513, 6, 128, 1024, 520),
    (4099, 32, 32, 264, 1096),
    # adapters without rows beside a gradient in one piece
    (20, 500, 8, 64, 264),
    (256, 300, 40, 520, 72),
    (300, 120, 8, 131080, 64),
    # few rows in one gradient's piece or several, and rows that are not few
    (1024, 9, 40, 520, 264),
    (1024, 2, 16, 136, 264),
    (1025, 9, 40, 520, 264),
    (777, 3, 96, 328, 72),
    (900, 1, 32, 72, 72),
    (384, 12, 16, 4096, 4096),
    (385, 12, 16, 4096, 4096),
]


@pytest.mark.parametrize("order", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_forward(gpu_ready, case, order):
    c = Case(*case, gap=8)
    c.forward(order)
    c.check_forward()


@pytest.mark.parametrize("case", CASES)
def test_backward(gpu_ready, case):
    c = Case(*case, gap=16, seed=1)
    c.forward()
    d_x = torch.full_like(c.dx_base, NAN)
    d_bank = torch.full((c.M, c.ad.stride), 7.0, device="cuda")
    c.backward(d_bank=d_bank, d_x=d_x, dx_base=c.dx_base)
    c.check_backward(d_x, d_bank)
    for m in c.mats(d_bank):
        m.fill_(7.0)
    assert (d_bank == 7.0).all()  # nothing but the windows was written


@pytest.mark.parametrize("case", [CASES[3], CASES[9], CASES[11], CASES[12]])
def test_accumulate_and_parts_alone(gpu_ready, case):
    c = Case(*case, seed=2)
    c.forward()
    old = torch.randn((c.M, c.ad.stride), generator=c.g, device="cuda")
    d_bank = old.clone()
    c.backward(accumulate=True, d_bank=d_bank)  # without d_x
    c.check_backward(None, d_bank, old)
    d_x = c.dx_base.clone()
    ws = c.work(True)
    mx.moonep_adapter_bwd(c.s, c.ad, c.ids, None, None, None, None, c.d_y, c.bank, c.scale, d_x, d_x, False, None, ws)
    c.check_backward(d_x, None)  # in place, without gradients, in the rows' own order


def test_in_place_gives_the_same_bits(gpu_ready):
    for case in (CASES[6], CASES[11], (9000, 5, 16, 1024, 264)):
        c = Case(*case)
        for order in (True, False):
            c.forward(order)
            y, u = c.y.clone(), c.u.clone()
            inplace = c.base.clone()
            c.forward(order, base=inplace, y=inplace)
            assert torch.equal(inplace, y) and torch.equal(c.u, u)
            c.y.copy_(y)
            c.check_forward()


@pytest.mark.parametrize("N", [40, 2200])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_an_adapter_of_nan_reaches_its_own_rows_only(gpu_ready, N, bad):
    c = Case(N, 5, 16, 64, 64, seed=3)
    c.forward(False)
    y, u = c.y.clone(), c.u.clone()
    d_x, d_bank = torch.empty_like(c.dx_base), torch.empty((5, c.ad.stride), device="cuda")
    c.backward(d_bank=d_bank, d_x=d_x, dx_base=c.dx_base)
    c.bank[2] = bad
    u0 = c.u.clone()
    c.forward(False)
    others = c.ids != 2
    assert torch.equal(c.y[others], y[others]) and torch.equal(c.u[others], u[others])
    assert not torch.isfinite(c.y[~others]).any()
    c.u = u0
    x2, b2 = torch.empty_like(d_x), torch.empty_like(d_bank)
    c.x[c.ids == 5] = NAN   # rows without an adapter are not looked at
    c.d_y[c.ids == 5] = NAN
    c.backward(d_bank=b2, d_x=x2, dx_base=c.dx_base)
    assert torch.equal(x2[others], d_x[others])
    keep = [0, 1, 3, 4]
    assert torch.equal(b2[keep], d_bank[keep])


def test_an_infinite_value_gives_an_infinity(gpu_ready):
    c = Case(20, 2, 8, 64, 64, none=0.0)
    A, B = c.mats(c.bank)
    c.x.zero_()
    c.x[3, 5] = float("inf")
    A.fill_(1.0)
    B.fill_(1.0)
    c.x[3, 5:6] = 3.0e38
    c.x[3, 6:7] = 3.0e38  # u of row 3 is beyond fp32
    c.forward()
    assert torch.isinf(c.u[3]).all() and torch.isinf(c.y[3]).all()
    rest = torch.arange(20, device="cuda") != 3
    assert torch.equal(c.y[rest], c.base[rest])


def test_gradients_are_the_forwards_differences(gpu_ready):
    """L = <d_y, y> in integers, exact: linear in x, A and B, one at a time."""
    c = Case(70, 4, 16, 64, 64, seed=4, integers=True)
    c.base.zero_()
    c.x[:, 8:].zero_()  # so that y stays below 257, exact in bf16
    c.d_y.clamp_(0, 1)
    A, B = c.mats(c.bank)
    B[:, :, 4:] = 0

    def loss():
        c.forward()
        assert c.y.abs().max() <= 256
        return (c.d_y.double() * c.y.double()).sum()

    L = loss()
    c.dx_base.zero_()
    d_x, d_bank = torch.empty_like(c.dx_base), torch.empty((4, c.ad.stride), device="cuda")
    c.backward(d_bank=d_bank, d_x=d_x, dx_base=c.dx_base)
    assert d_x.abs().max() <= 256
    dA, dB = c.mats(d_bank)
    one = lambda t: torch.randint(-1, 2, t.shape, generator=c.g, device="cuda").bfloat16()  # noqa: E731
    for t, grad in ((A, dA), (B, dB), (c.x, d_x)):
        was, step = t.clone(), one(t)
        if t is c.x:
            step[:, 8:] = 0
        if t is B:
            step[:, :, 4:] = 0
        t += step
        assert loss() - L == (grad.double() * step.double()).sum()
        t.copy_(was)


def test_adapters_without_rows_and_no_rows(gpu_ready):
    c = Case(40, 6, 16, 64, 64, seed=5)
    c.ids.fill_(6)
    c.ids[:10] = 4
    mx.plan_step(c.b, c.ids)
    c.forward()
    old = torch.ones((6, c.ad.stride), device="cuda")
    d_bank = old.clone()
    c.backward(accumulate=True, d_bank=d_bank)
    assert (d_bank[[0, 1, 2, 3, 5]] == 1).all() and not (d_bank[4] == 1).all()
    c.backward(d_bank=d_bank)
    assert (d_bank[[0, 1, 2, 3, 5]] == 0).all()
    e = Case(0, 3, 8, 64, 64)
    e.forward()
    d_bank = torch.ones((3, e.ad.stride), device="cuda")
    e.backward(accumulate=True, d_bank=d_bank)
    assert (d_bank == 1).all()
    e.backward(d_bank=d_bank, d_x=e.dx_base, dx_base=e.dx_base)
    assert (d_bank == 0).all()


def test_one_adapter_over_many_chunks_and_long_runs(gpu_ready):
    for N, M, runs in ((9000, 1, None), (8200, 2, 4100), (6000, 12, 500)):
        c = Case(N, M, 8, 64, 72, none=0.0 if M < 3 else 0.1, seed=6, runs=runs)
        c.forward()
        c.check_forward()
        d_x, d_bank = torch.empty_like(c.dx_base), torch.empty((M, c.ad.stride), device="cuda")
        c.backward(d_bank=d_bank, d_x=d_x, dx_base=c.dx_base)
        c.check_backward(d_x, d_bank)
        again = torch.empty_like(d_bank)
        c.backward(d_bank=again)
        assert torch.equal(again, d_bank)  # no sum depends on timing


def test_tables_of_another_plan_stay_in_bounds(gpu_ready):
    """Order and plan that do not belong to the ids: the windows only are written."""
    c = Case(300, 4, 16, 64, 64, gap=8, seed=7)
    c.forward()
    d_bank = torch.full((4, c.ad.stride), 7.0, device="cuda")
    c.order = torch.randint(-5, 310, (300,), generator=c.g, device="cuda").int()
    c.plan = torch.randint(-1000, 1000, c.plan.shape, generator=c.g, device="cuda").int()
    d_x = c.dx_base.clone()
    c.backward(d_bank=d_bank, d_x=d_x, dx_base=c.dx_base)
    c.forward()
    torch.cuda.synchronize()
    for m in c.mats(d_bank):
        m.fill_(7.0)
    assert (d_bank == 7.0).all()


def test_graph_and_streams(gpu_ready):
    """Both directions captured and replayed over new inputs, and two at once on
    two streams, each with its own workspace."""
    cs = [Case(333, 5, 16, 128, 136, seed=8), Case(2300, 5, 16, 128, 136, seed=9)]
    outs = [(torch.empty_like(c.dx_base), torch.empty((5, c.ad.stride), device="cuda")) for c in cs]
    works = [(c.work(), c.work(True)) for c in cs]

    def step(c, o, w):
        c.forward(ws=w[0])
        c.backward(d_bank=o[1], d_x=o[0], dx_base=c.dx_base, ws=w[1])

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for st, c, o, w in zip(streams, cs, outs, works):
        with torch.cuda.stream(st):
            step(c, o, w)
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        c.check_forward()
        c.check_backward(*o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o, w in zip(cs, outs, works):
            step(c, o, w)
    for k in range(3):
        for c in cs:
            c.x.copy_(torch.randn(c.x.shape, generator=c.g, device="cuda").bfloat16())
            c.d_y.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        for c, o in zip(cs, outs):
            c.check_forward()
            c.check_backward(*o)
