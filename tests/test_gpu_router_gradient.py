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
