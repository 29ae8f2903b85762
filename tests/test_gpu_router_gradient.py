"""The router's backward where its terms cancel: one chosen expert, one that dominates, counts that are nearly equal.

The normalised gates' term is dg_k - sum_j dg_j s_j / W and the loss's a_e - sum_j a_j p_j.  Neither changes when a
constant comes off every dg or every a, but for d tiny / W (a tiny / Z) of it with sigmoid, whose W and Z hold
tiny = 1e-20 besides the scores.  So a sound backward owes errors relative to what is left after the token's first
d_gates, and a group's mean count, have come off: a zero there is a zero, and the rest is not the rounding noise of
terms that cancel.

Bounds: each such term is a product of a few factors, every one of them within ref.rel of its true value (see
test_gpu_router.py), its sums of K entries within K 2^-24, so 4 ref.rel + (K + 16) 2^-24 of the magnitudes left;
then half a step of the output's type.  Rounded to integers, the mean count is half a count off: |a| grows by it."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx
from gpu_harness import to_dev
from test_gpu_router import SIG, SOFT, Ref, as_type, order

pytestmark = pytest.mark.gpu


def left(ref, dg, dl, T):
    """d_logits in 64 bits from the terms left after the shifts, and the sum of their magnitudes."""
    o, K, E = ref.o, ref.ids.shape[1], ref.l.shape[1]
    tiny = 1e-20 if o.score == SIG else 0.0
    slope = ref.s if o.score == SOFT else ref.s * (1 - ref.s)
    factor = dl * E / (K * float(ref.n) ** 2 * ref.G)
    mean = ref.n * K / E
    a = np.repeat(factor * (T - mean), ref.n, 0)
    mag_a = np.repeat(abs(factor) * (np.abs(T - mean) + 0.5), ref.n, 0)
    a0, mag_a0 = factor * mean * tiny * ref.rz, abs(factor) * (mean + 0.5) * tiny * ref.rz
    ds = (a - (a * ref.p).sum(1, keepdims=True) + a0) * ref.rz
    mag = (mag_a + (mag_a * ref.p).sum(1, keepdims=True) + mag_a0) * ref.rz
    d0 = dg[:, :1]
    d = dg - d0
    s = np.take_along_axis(ref.s, ref.ids, 1)
    part = (d - (d * s).sum(1, keepdims=True) * ref.rw + d0 * tiny * ref.rw) * o.scale * ref.rw
    part_mag = (np.abs(d) + (np.abs(d) * s).sum(1, keepdims=True) * ref.rw + np.abs(d0) * tiny * ref.rw) * abs(o.scale) * ref.rw
    full, full_mag = np.zeros_like(ds), np.zeros_like(ds)
    np.put_along_axis(full, ref.ids, part, 1)
    np.put_along_axis(full_mag, ref.ids, part_mag, 1)
    return (ds + full) * slope, (mag + full_mag) * slope


def backward(shape, opts, d, ids, T, dg, dl):
    """d_logits for the given ids and counts; dg or dl None: without the gates, or the loss."""
    out = torch.full_like(d, float("nan"))
    mx.moonep_router_bwd(shape, opts, d, to_dev(ids.reshape(-1)), None if dl is None else to_dev(T.astype(np.int32)),
                         None if dg is None else to_dev(dg.reshape(-1)),
                         None if dl is None else to_dev(np.array([dl], np.float32)), out)
    torch.cuda.synchronize()
    return out.double().cpu().numpy()


def check(got, want, mag, ref, bf16):
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    err = mag * (4 * ref.rel + (ref.ids.shape[1] + 16) * 2.0 ** -24) + 2.0 ** -126
    off = np.abs(got - want)
    allowed = np.abs(want) * half + err
    assert (off <= allowed).all(), f"{(off / allowed).max()} of what is allowed"


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
def test_one_chosen_expert_normalised(score, bf16):
    """The gate is the constant `scale`: no gradient with softmax, and with sigmoid what tiny leaves."""
    rng = np.random.default_rng(21)
    for N, E, spread in ((700, 16, 1.0), (33, 1, 1.0), (129, 130, 4.0)):
        print(f"[case] K=1 N={N} E={E} score={score} bf16={bf16}", flush=True)
        t = as_type(spread * rng.standard_normal((N, E)), bf16)
        l = t.double().numpy()
        opts = mx.RouterOpts(score, True, 1, int(bf16), 2.5)
        ids = order(l, 1)
        dg = rng.standard_normal((N, 1)).astype(np.float32)
        got = backward(mx.Shape(1, E, N, 1, 16), opts, t.cuda(), ids, None, dg, None)
        if score == SOFT:
            assert (got == 0).all()
            continue
        s = np.take_along_axis(1 / (1 + np.exp(-l)), ids, 1)
        allowed = np.zeros((N, E))
        np.put_along_axis(allowed, ids, 2.5 * np.abs(dg) * 1e-20 / (s + 1e-20) ** 2 * s * (1 - s), 1)
        assert (np.abs(got) <= 1.01 * allowed + 2.0 ** -126).all()


# tokens, experts, K, groups, score, factor of the gates, how far the first choice stands above the others
TRAINING = [
    ("k1", 7300, 16, 1, 1, SIG, 2.5, 0.0),
    ("k1_wide", 32768, 64, 1, 1, SIG, 2.5, 0.0),
    ("k1_two", 65536, 2, 1, 1, SIG, 1.0, 0.0),
    ("k1_softmax", 8192, 64, 1, 4, SOFT, 1.0, 0.0),
    ("dominant", 4096, 64, 8, 1, SIG, 1.0, 17.0),
    ("dominant_softmax", 4096, 130, 6, 2, SOFT, 2.5, 17.0),
    ("many_chosen", 2048, 64, 20, 1, SIG, 1.0, 16.0),
    ("even", 16384, 32, 4, 8, SOFT, 1.0, 0.0),
]


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", TRAINING, ids=lambda c: c[0])
def test_training_proportions(case, bf16):
    """d_gates of 0.1 beside a loss weight of 0.01, spread over all tokens: the loss's gradient is far below
    2^-24 of a single gate's."""
    name, N, E, K, G, score, scale, above = case
    print(f"[case] {name} bf16={bf16}", flush=True)
    rng = np.random.default_rng(22)
    l = rng.standard_normal((N, E)) - above
    l[np.arange(N), rng.integers(0, E, N)] += 2 * above if score == SIG else above
    t = as_type(l, bf16)
    l = t.double().numpy()
    ids = order(l, K)
    opts = mx.RouterOpts(score, True, G, int(bf16), scale)
    ref = Ref(l, ids, opts, G)
    dg = (0.1 * rng.standard_normal((N, K))).astype(np.float32)
    dl = np.float32(0.01)
    for use in (dg, np.zeros_like(dg)):
        got = backward(mx.Shape(1, E, N, K, 16), opts, t.cuda(), ids, ref.T, use, dl)
        check(got, *left(ref, use.astype(np.float64), float(dl), ref.T), ref, bf16)


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
def test_even_counts(score):
    """Counts that are all equal leave no gradient of the loss (with sigmoid, tiny's); counts a few apart leave theirs."""
    rng = np.random.default_rng(23)
    N, E, K = 4096, 64, 8
    t = as_type(rng.standard_normal((N, E)), False)
    l = t.double().numpy()
    ids = order(l, K)
    opts = mx.RouterOpts(score, False, 1, mx.F32, 1.0)
    ref = Ref(l, ids, opts, 1)
    shape = mx.Shape(1, E, N, K, 16)
    T = np.full((1, E), N * K // E)
    got = backward(shape, opts, t.cuda(), ids, T, None, 1.0)
    if score == SOFT:
        assert (got == 0).all()
    else:
        assert np.abs(got).max() <= 1e-20
    T = T + rng.integers(-2, 3, (1, E))
    zero = np.zeros((N, K))
    check(backward(shape, opts, t.cuda(), ids, T, None, 1.0), *left(ref, zero, 1.0, T), ref, False)


def test_first_id_refused_normalised():
    """A token whose first ids are outside [0, E): they contribute nothing, the others as if alone."""
    rng = np.random.default_rng(24)
    N, E, K = 40, 20, 4
    t = as_type(rng.standard_normal((N, E)), False)
    l = t.double().numpy()
    ids = order(l, K)
    dg = rng.standard_normal((N, K)).astype(np.float32)
    bad = ids.copy()
    bad[::3, 0], bad[1::5, 1], bad[7] = -1, E, E + 3
    for score in (SOFT, SIG):
        opts = mx.RouterOpts(score, True, 1, mx.F32, 1.5)
        got = backward(mx.Shape(1, E, N, K, 16), opts, t.cuda(), bad, None, dg, None)
        s = np.exp(l - l.max(1, keepdims=True)) if score == SOFT else 1 / (1 + np.exp(-l))
        slope = s if score == SOFT else s * (1 - s)
        ok = (bad >= 0) & (bad < E)
        sk = np.where(ok, np.take_along_axis(s, np.where(ok, bad, 0), 1), 0)
        W = sk.sum(1, keepdims=True)
        W[W == 0] = 1
        want, mag = np.zeros((N, E)), np.zeros((N, E))
        for out, v in ((want, dg - (dg * sk).sum(1, keepdims=True) / W),
                       (mag, np.abs(dg) + (np.abs(dg) * sk).sum(1, keepdims=True) / W)):
            for k in range(K):
                np.add.at(out, (np.arange(N), np.where(ok[:, k], bad[:, k], 0)), np.where(ok, 1.5 * v / W, 0)[:, k])
        rel = (2 * np.abs(l - l.max(1, keepdims=True)).max() + E / 8 + 32) * 2.0 ** -24
        allowed = (np.abs(want) * 2.0 ** -24 + mag * (4 * rel + (K + 16) * 2.0 ** -24)) * slope + 2.0 ** -126
        assert (np.abs(got - want * slope) <= allowed).all()
