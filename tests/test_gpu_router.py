"""The router on the GPU -- ids, gates, counts, balance loss and their gradient --
against its definition in 64 bits.

Bounds.  With X the largest |logit - top| of a row (softmax) or |logit|
(sigmoid), the fp32 scores are within (2 X + 8) 2^-24 of the true ones relative:
the subtraction's rounding X 2^-24, the exponential's few units.  A sum of them
over E experts adds at most (E / 16 + 8) 2^-24, and each further operation 2^-24."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx
from gpu_harness import to_dev

pytestmark = pytest.mark.gpu

SOFT, SIG = mx.SCORE_SOFTMAX, mx.SCORE_SIGMOID


def as_type(l, bf16):
    t = torch.from_numpy(np.ascontiguousarray(l, dtype=np.float32))
    return t.to(torch.bfloat16) if bf16 else t


def order(l, K):
    """ids of the K largest of each row, descending, ties to the lower id."""
    return np.argsort(-l, axis=1, kind="stable")[:, :K].astype(np.int32)


class Ref:
    """Definition in 64 bits, for logits l [N, E] and given ids."""

    def __init__(self, l, ids, opts, n_groups):
        self.l, self.ids, self.o = l, ids, opts
        N, E = l.shape
        tiny = 1e-20 if opts.score == SIG else 0.0
        with np.errstate(all="ignore"):
            if opts.score == SOFT:
                top = l.max(1, keepdims=True)
                self.x = np.where(np.isinf(l), 0, l - np.where(np.isinf(top), 0, top))
                self.s = np.exp(l - np.where(np.isinf(top), 0, top))
            else:
                self.x = np.where(np.isinf(l), 0, l)
                self.s = 1 / (1 + np.exp(-l))
            self.Z = self.s.sum(1, keepdims=True) + tiny
            self.rz = np.where(self.Z == 0, 0, 1 / self.Z)
        self.p = self.s * self.rz
        top_s = np.take_along_axis(self.s, ids, 1)
        self.W = top_s.sum(1, keepdims=True) + tiny
        with np.errstate(all="ignore"):
            self.rw = np.where(self.W == 0, 0, 1 / self.W)
        self.mul = self.rw if opts.normalize else (self.rz if opts.score == SOFT else np.ones_like(self.Z))
        self.gates = opts.scale * top_s * self.mul
        self.G = n_groups
        self.n = N // n_groups
        self.T = np.stack([np.bincount(ids[g * self.n:(g + 1) * self.n].ravel(), minlength=E) for g in range(n_groups)])
        self.P = self.p.reshape(n_groups, self.n, E).sum(1)
        self.loss = (self.T * self.P).sum() * E / (ids.shape[1] * self.n ** 2 * n_groups) if self.n else 0.0
        self.rel = (2 * np.abs(self.x).max(initial=0) + E / 8 + 32) * 2.0 ** -24

    def grad(self, dg, dl):
        """d_logits, and the sum of its terms' magnitudes."""
        N, E = self.l.shape
        K = self.ids.shape[1]
        a = np.repeat(dl * E / (K * self.n ** 2 * self.G) * self.T, self.n, axis=0)
        dot = (a * self.p).sum(1, keepdims=True)
        ds, mag = (a - dot) * self.rz, (a + dot) * self.rz
        full, chosen = np.zeros((N, E)), np.zeros((N, E))
        np.put_along_axis(full, self.ids, dg, 1)
        np.put_along_axis(chosen, self.ids, 1.0, 1)
        c = self.o.scale
        if self.o.normalize:
            sub = (full * self.s).sum(1, keepdims=True) * self.rw
            suba = (np.abs(full) * self.s).sum(1, keepdims=True) * self.rw
            ds = ds + c * self.rw * chosen * (full - sub)
            mag = mag + c * self.rw * chosen * (np.abs(full) + suba)
        elif self.o.score == SOFT:
            ds = ds + c * self.rz * (full - (full * self.p).sum(1, keepdims=True))
            mag = mag + c * self.rz * (np.abs(full) + (np.abs(full) * self.p).sum(1, keepdims=True))
        else:
            ds, mag = ds + c * full, mag + c * np.abs(full)
        slope = self.s if self.o.score == SOFT else self.s * (1 - self.s)
        return ds * slope, mag * slope


def forward(shape, opts, logits, loss=True, fill=-5):
    dev = "cuda"
    out = dict(ids=torch.full((shape.NK,), fill, dtype=torch.int32, device=dev),
               gates=torch.full((shape.NK,), float(fill), device=dev))
    if loss:
        out.update(counts=torch.full((opts.groups, shape.E), fill, dtype=torch.int32, device=dev),
                   prob_sum=torch.full((opts.groups, shape.E), float(fill), device=dev),
                   loss=torch.full((1,), float(fill), device=dev))
        ws = torch.full((mx.moonep_router_workspace_bytes(shape, opts),), 0xEE, dtype=torch.uint8, device=dev)
        mx.moonep_router(shape, opts, logits, out["ids"], out["gates"], out["counts"], out["prob_sum"], out["loss"], ws)
    else:
        mx.moonep_router(shape, opts, logits, out["ids"], out["gates"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def logits_for(rng, N, E, bf16, spread=1.0):
    l = spread * (rng.standard_normal((N, E)) + 0.5 * rng.standard_normal(E))
    t = as_type(l, bf16)
    return t, t.double().numpy()


SHAPES = [
    # R, E, S, K, groups
    (1, 1, 1, 1, 1), (1, 8, 1, 2, 1), (2, 10, 9, 3, 2), (1, 60, 33, 4, 3), (4, 64, 16, 8, 4), (3, 66, 7, 6, 21),
    (2, 128, 130, 8, 1), (1, 130, 5, 1, 1), (8, 256, 40, 8, 8), (1, 257, 19, 17, 1), (2, 512, 11, 32, 2),
    (1, 1023, 6, 8, 1), (4, 1024, 5, 16, 4), (1, 20, 12, 20, 1), (1, 64, 5000, 2, 1), (1, 40, 37, 40, 1),
]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("R,E,S,K,groups", SHAPES)
def test_forward_and_backward(R, E, S, K, groups, score, bf16):
    rng = np.random.default_rng(E * 7 + S)
    shape = mx.Shape(R, E, S, K, 16)
    for normalize, scale in ((True, 2.5), (False, 1.0)):
        print(f"[case] router R={R} E={E} S={S} K={K} G={groups} score={score} bf16={bf16} norm={normalize}", flush=True)
        opts = mx.RouterOpts(score, normalize, groups, int(bf16), scale)
        t, l = logits_for(rng, R * S, E, bf16)
        ids = order(l, K)
        ref = Ref(l, ids, opts, groups)
        d = t.cuda()
        got = forward(shape, opts, d)
        np.testing.assert_array_equal(got["ids"].reshape(-1, K), ids)
        np.testing.assert_allclose(got["gates"].reshape(-1, K), ref.gates, rtol=2 * ref.rel, atol=0)
        np.testing.assert_array_equal(got["counts"], ref.T)
        rel = 2 * ref.rel + (ref.n / 16 + 16) * 2.0 ** -24
        np.testing.assert_allclose(got["prob_sum"], ref.P, rtol=rel, atol=0)
        np.testing.assert_allclose(got["loss"][0], ref.loss, rtol=rel + 2.0 ** -23)
        bare = forward(shape, opts, d, loss=False)
        for k in ("ids", "gates"):
            np.testing.assert_array_equal(bare[k], got[k])

        dg = rng.standard_normal((R * S, K)).astype(np.float32)
        dl = np.float32(0.37)
        d_l = torch.full_like(d, float("nan"))
        counts = to_dev(got["counts"])
        for use_g, use_l in ((True, True), (True, False), (False, True)):
            mx.moonep_router_bwd(shape, opts, d, to_dev(got["ids"]), counts if use_l else None,
                                 to_dev(dg.reshape(-1)) if use_g else None,
                                 to_dev(np.array([dl])) if use_l else None, d_l)
            torch.cuda.synchronize()
            want, mag = ref.grad(dg.astype(np.float64) * use_g, float(dl) * use_l)
            half = 2.0 ** -8 if bf16 else 2.0 ** -24
            allowed = np.abs(want) * half + mag * (4 * ref.rel + (K + 16) * 2.0 ** -24) + 2.0 ** -126
            off = np.abs(d_l.double().cpu().numpy() - want)
            assert (off <= allowed).all(), f"{(off / allowed).max()} of what is allowed"


@pytest.mark.parametrize("score,normalize", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
def test_gradient_against_differences(score, normalize):
    """Central differences of the definition in 64 bits, step h: the error of a
    difference is h^2/6 of the third derivative plus rounding 2^-52/h, both under
    1e-7 here for h = 1e-4 (terms of order 1)."""
    rng = np.random.default_rng(5)
    R, E, S, K, G, h = 2, 12, 3, 3, 2, 1e-4
    opts = mx.RouterOpts(score, normalize, G, mx.F32, 1.5)
    t, l = logits_for(rng, R * S, E, False)
    ids = order(l, K)
    dg, dl = rng.standard_normal((R * S, K)).astype(np.float32), np.float32(0.8)
    T = Ref(l, ids, opts, G).T

    def total(v):
        r = Ref(v, ids, opts, G)
        n = r.n
        return (r.gates * dg).sum() + float(dl) * (T * r.P).sum() * E / (K * n * n * G)

    want = np.zeros_like(l)
    for i in range(l.shape[0]):
        for e in range(E):
            v = l.copy()
            v[i, e] += h
            up = total(v)
            v[i, e] -= 2 * h
            want[i, e] = (up - total(v)) / (2 * h)
    d_l = torch.empty((R * S, E), device="cuda")
    mx.moonep_router_bwd(mx.Shape(R, E, S, K, 16), opts, t.cuda(), to_dev(ids.reshape(-1)), to_dev(T.astype(np.int32)),
                         to_dev(dg.reshape(-1)), to_dev(np.array([dl])), d_l)
    torch.cuda.synchronize()
    np.testing.assert_allclose(d_l.cpu().numpy(), want, rtol=1e-5, atol=5e-6)


def test_ties_go_to_the_lower_id():
    """Few distinct values, +0 and -0 among them."""
    rng = np.random.default_rng(6)
    for E, K in ((8, 8), (64, 8), (100, 20), (256, 8), (1000, 5)):
        print(f"[case] ties E={E} K={K}", flush=True)
        l = rng.integers(-2, 3, (50, E)).astype(np.float32)
        l[l == 0] = np.where(rng.random((l == 0).sum()) < 0.5, -0.0, 0.0)
        for bf16 in (False, True):
            got = forward(mx.Shape(1, E, 50, K, 16), mx.RouterOpts(SOFT, True, 1, int(bf16)), as_type(l, bf16).cuda())
            np.testing.assert_array_equal(got["ids"].reshape(50, K), order(l.astype(np.float64) + 0.0, K))


def test_near_ties():
    """Neighbouring fp32 values, which differ in the last bit alone."""
    rng = np.random.default_rng(7)
    base = np.float32(1.2345).view(np.int32)
    for E in (16, 64, 256):
        l = (base + rng.integers(0, E, (64, E)).astype(np.int32)).view(np.float32) * np.where(rng.random((64, 1)) < 0.5, 1, -1).astype(np.float32)
        got = forward(mx.Shape(1, E, 64, 8, 16), mx.RouterOpts(SOFT, False), torch.from_numpy(l).cuda())
        np.testing.assert_array_equal(got["ids"].reshape(64, 8), order(l.astype(np.float64), 8))


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("low", [-np.inf, np.finfo(np.float32).min])
def test_masked_experts(score, low):
    """Experts masked by -inf or the type's lowest value; a token with nothing left.  With -inf on all, gates and shares
    are 0; with the lowest value on all, softmax has equal shares."""
    rng = np.random.default_rng(8)
    R, E, S, K = 2, 24, 8, 4
    l = rng.standard_normal((R * S, E)).astype(np.float32)
    l[rng.random((R * S, E)) < 0.6] = low
    l[3] = low
    l[4, 1:] = low
    for normalize in (True, False):
        print(f"[case] masked score={score} low={low} norm={normalize}", flush=True)
        opts = mx.RouterOpts(score, normalize, 2, mx.F32, 1.0)
        shape = mx.Shape(R, E, S, K, 16)
        d = torch.from_numpy(l).cuda()
        got = forward(shape, opts, d)
        ids = order(l.astype(np.float64), K)
        np.testing.assert_array_equal(got["ids"].reshape(-1, K), ids)
        lf = l.astype(np.float64)
        ref = Ref(lf, ids, opts, 2)
        ok = np.where(lf < -1e30, 0, np.abs(lf)).max()
        rel = (4 * ok + 80) * 2.0 ** -24
        np.testing.assert_allclose(got["gates"].reshape(-1, K), ref.gates, rtol=rel, atol=1e-30)
        np.testing.assert_allclose(got["prob_sum"], ref.P, rtol=2 * rel, atol=1e-30)
        np.testing.assert_array_equal(got["counts"], ref.T)
        if low == -np.inf:
            assert (got["gates"].reshape(-1, K)[3] == 0).all()
        dg = rng.standard_normal((R * S, K)).astype(np.float32)
        d_l = torch.full_like(d, float("nan"))
        mx.moonep_router_bwd(shape, opts, d, to_dev(got["ids"]), to_dev(got["counts"]), to_dev(dg.reshape(-1)),
                             torch.ones(1, device="cuda"), d_l)
        torch.cuda.synchronize()
        want, mag = ref.grad(dg.astype(np.float64), 1.0)
        off = np.abs(d_l.double().cpu().numpy() - want)
        assert (off <= mag * 8 * rel + np.abs(want) * 2.0 ** -24 + 1e-30).all()


def test_non_finite_logits():
    """NaN ranks last, and the ids stay distinct and valid; other rows keep their results."""
    rng = np.random.default_rng(9)
    N, E, K = 40, 30, 6
    l = rng.standard_normal((N, E)).astype(np.float32)
    clean = forward(mx.Shape(1, E, N, K, 16), mx.RouterOpts(SOFT, False), torch.from_numpy(l).cuda(), loss=False)
    l[5, 3] = np.nan
    l[6, :] = np.nan
    l[7, 2:] = np.nan
    l[9, 4] = np.inf
    got = forward(mx.Shape(1, E, N, K, 16), mx.RouterOpts(SOFT, False), torch.from_numpy(l).cuda(), loss=False)
    ids, gates = got["ids"].reshape(N, K), got["gates"].reshape(N, K)
    assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == K for r in ids.tolist())
    assert 3 not in ids[5] and ids[6].tolist() == list(range(K)) and set(ids[7][:2]) == {0, 1} and ids[9][0] == 4
    assert np.isnan(gates[[5, 6, 7, 9]]).any(1).all()
    rest = np.setdiff1d(np.arange(N), [5, 6, 7, 9])
    np.testing.assert_array_equal(ids[rest], clean["ids"].reshape(N, K)[rest])
    np.testing.assert_array_equal(gates[rest], clean["gates"].reshape(N, K)[rest])


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
def test_wide_logits(score):
    """Logits of +-60: scores from 1 down to 1e-52 (0 in fp32)."""
    rng = np.random.default_rng(10)
    l = (rng.random((64, 48)) * 120 - 60).astype(np.float32)
    opts = mx.RouterOpts(score, True, 1, mx.F32, 1.0)
    got = forward(mx.Shape(1, 48, 64, 8, 16), opts, torch.from_numpy(l).cuda())
    ref = Ref(l.astype(np.float64), order(l.astype(np.float64), 8), opts, 1)
    np.testing.assert_array_equal(got["ids"].reshape(64, 8), ref.ids)
    np.testing.assert_allclose(got["gates"].reshape(64, 8), ref.gates, rtol=2 * ref.rel, atol=2.0 ** -120)
    np.testing.assert_allclose(got["loss"][0], ref.loss, rtol=2 * ref.rel)


def test_counts_agree_with_route_stats_and_empty():
    rng = np.random.default_rng(11)
    s = mx.Shape(4, 32, 77, 4, 16)
    t, _ = logits_for(rng, s.N, s.E, False)
    b = mx.allocate(s)
    got = forward(s, mx.RouterOpts(SOFT, True, 1), t.cuda())
    mx.plan_step(b, to_dev(got["ids"]))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(b.expert_counts.cpu().numpy(), got["counts"][0])
    assert mx.moonep_read_error(b.workspace) == 0
    e = mx.Shape(4, 32, 0, 4, 16)
    got = forward(e, mx.RouterOpts(SOFT, True, 4), torch.empty((0, 32), device="cuda"))
    assert (got["counts"] == 0).all() and (got["prob_sum"] == 0).all() and got["loss"][0] == 0


def test_same_bits_every_time():
    rng = np.random.default_rng(12)
    s, opts = mx.Shape(8, 64, 3001, 8, 16), mx.RouterOpts(SOFT, True, 1)
    t, _ = logits_for(rng, s.N, s.E, False)
    d = t.cuda()
    first = forward(s, opts, d)
    for _ in range(3):
        again = forward(s, opts, d)
        for k in first:
            np.testing.assert_array_equal(first[k].view(np.int32), again[k].view(np.int32), err_msg=k)


def test_backward_ignores_bad_ids():
    """Ids outside [0, E) contribute nothing; the same id twice counts twice."""
    rng = np.random.default_rng(13)
    N, E, K = 6, 16, 4
    s, opts = mx.Shape(1, E, N, K, 16), mx.RouterOpts(SIG, False, 1)
    t, l = logits_for(rng, N, E, False)
    ids = order(l, K)
    ids[0, 1], ids[2, 3] = -1, E
    ids[4] = [7, 7, 2, 7]
    dg = rng.standard_normal((N, K)).astype(np.float32)
    d_l = torch.empty((N, E), device="cuda")
    mx.moonep_router_bwd(s, opts, t.cuda(), to_dev(ids.reshape(-1)), None, to_dev(dg.reshape(-1)), None, d_l)
    torch.cuda.synchronize()
    want = np.zeros((N, E))
    mag = np.zeros((N, E))
    for i in range(N):
        for k in range(K):
            if 0 <= ids[i, k] < E:
                want[i, ids[i, k]] += dg[i, k]
                mag[i, ids[i, k]] += abs(dg[i, k])
    sg = 1 / (1 + np.exp(-l))
    off = np.abs(d_l.double().cpu().numpy() - want * sg * (1 - sg))
    assert (off <= mag * sg * (1 - sg) * (2 * np.abs(l).max() + 40) * 2.0 ** -24).all()


def test_shared_leading_bits():
    """fp32 logits that agree in the leading bits the fast rounds compare: at the border of the chosen, among them, in
    one row of a wave, and with a NaN elsewhere."""
    rng = np.random.default_rng(14)
    for E, K in ((40, 4), (128, 8), (256, 8), (512, 20), (1024, 8)):
        print(f"[case] leading bits E={E} K={K}", flush=True)
        l = rng.standard_normal((37, E)).astype(np.float32)
        for i in range(0, 37, 3):
            # a cluster of K + 2 values around 3, in the last bits only, in random places
            at = rng.permutation(E)[:K + 2]
            l[i, at] = (np.float32(3).view(np.int32) + rng.integers(0, 3, at.size).astype(np.int32)).view(np.float32)
        for i in range(1, 37, 6):
            o = np.argsort(-l[i])
            l[i, o[K]] = l[i, o[K - 1]]  # the border alone
        for score in (SOFT, SIG):
            got = forward(mx.Shape(1, E, 37, K, 16), mx.RouterOpts(score, True), torch.from_numpy(l).cuda())
            np.testing.assert_array_equal(got["ids"].reshape(37, K), order(l.astype(np.float64), K))


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_unaligned_logits(bf16):
    """Rows that start on no vector: logits and d_logits one element into their allocations."""
    rng = np.random.default_rng(15)
    s, opts = mx.Shape(2, 64, 21, 6, 16), mx.RouterOpts(SOFT, True, 2, int(bf16))
    t, l = logits_for(rng, s.N, s.E, bf16)
    dg = to_dev(rng.standard_normal(s.NK).astype(np.float32))

    def both(shift):
        buf = torch.zeros(s.N * s.E + 8, dtype=t.dtype, device="cuda")
        out = torch.full_like(buf, float("nan"))
        d, o = buf[shift:shift + s.N * s.E].view(s.N, s.E), out[shift:shift + s.N * s.E].view(s.N, s.E)
        d.copy_(t)
        got = forward(s, opts, d)
        mx.moonep_router_bwd(s, opts, d, to_dev(got["ids"]), to_dev(got["counts"]), dg, torch.ones(1, device="cuda"), o)
        torch.cuda.synchronize()
        assert torch.isnan(out[:shift]).all() and torch.isnan(out[shift + s.N * s.E:]).all()
        return got, o.float().cpu().numpy()

    a, b = both(0), both(1)
    for k in a[0]:
        np.testing.assert_array_equal(a[0][k], b[0][k], err_msg=k)
    np.testing.assert_array_equal(a[1], b[1])


def test_logits_far_into_memory():
    """More than 2^31 elements of logits: offsets past 32 bits, checked on the last rows."""
    s, opts = mx.Shape(1, 1024, (1 << 21) + 77, 2, 16), mx.RouterOpts(SOFT, False, 1, mx.BF16)
    d = torch.zeros((s.N, s.E), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1 << 20, s.N - 2, s.N - 1]
    rng = np.random.default_rng(16)
    v = rng.standard_normal((len(rows), s.E)).astype(np.float32)
    for r, x in zip(rows, v):
        d[r] = torch.from_numpy(x).cuda()
    ids = torch.empty(s.NK, dtype=torch.int32, device="cuda")
    gates = torch.empty(s.NK, device="cuda")
    mx.moonep_router(s, opts, d, ids, gates)
    d_l = torch.empty_like(d)
    dg = torch.ones(s.NK, device="cuda")
    mx.moonep_router_bwd(s, opts, d, ids, None, dg, None, d_l)
    torch.cuda.synchronize()
    l = d[rows].double().cpu().numpy()
    want = order(l, 2)
    np.testing.assert_array_equal(ids.view(-1, 2)[rows].cpu().numpy(), want)
    assert (ids.view(-1, 2)[5].cpu().numpy() == [0, 1]).all()
    ref = Ref(l, want, opts, 1)
    np.testing.assert_allclose(gates.view(-1, 2)[rows].cpu().numpy(), ref.gates, rtol=2 * ref.rel)
    g, mag = ref.grad(np.ones((len(rows), 2)), 0.0)
    off = np.abs(d_l[rows].double().cpu().numpy() - g)
    assert (off <= np.abs(g) * 2.0 ** -8 + mag * (4 * ref.rel + 32 * 2.0 ** -24) + 2.0 ** -126).all()
