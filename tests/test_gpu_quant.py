"""The 8-bit path on the GPU -- norm, dispatch, weights, products -- against
64-bit references: exact where the operator only rounds or copies, within bounds
that count each rounding otherwise.

Rounding of an fp32 value to bf16 is at most 2^-8 of it (half a step), an fp32
operation 2^-24.  An fp32 sum of n terms is at most n 2^-23 of the sum of their
magnitudes off, in any order."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx
import oracle
import synth
from gpu_harness import bf16_dev, bits, oracle_plan, shape_of, to_dev
from quant_ref import (check_rows, expand, host, quantise, scale_bytes, scale_of, values,
                       weight_values)

pytestmark = pytest.mark.gpu


def f64(b):
    return (np.asarray(b, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_of(v):
    t = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def codes_dev(a):
    return to_dev(a).view(torch.float8_e4m3fn)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def run_norm(x, res, w, eps, want_y=True, inplace=False):
    N, H = x.shape
    dx, dr = bf16_dev(x), None if res is None else bf16_dev(res)
    out = None if res is None else (dr if inplace else torch.full_like(dx, float("nan")))
    y = torch.full_like(dx, float("nan")) if want_y else None
    y8 = torch.full((N, H), 0x55, dtype=torch.uint8, device="cuda")
    ys = torch.full((N, scale_bytes(H)), 0x55, dtype=torch.uint8, device="cuda")
    mx.moonep_rmsnorm_quant(mx.Shape(1, 1, N, 1, H), dx, dr, bf16_dev(w), eps, out, y, y8, ys)
    torch.cuda.synchronize()
    return out, y, host(y8), host(ys)


def check_norm(x, res, w, eps, inplace=False):
    N, H = x.shape
    out, y, y8, ys = run_norm(x, res, w, eps, inplace=inplace)
    r = x if res is None else bf16_of(f64(x).astype(np.float32) + f64(res).astype(np.float32))
    if res is not None:
        np.testing.assert_array_equal(bits(out), r)
    v = f64(r)
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * f64(w)
    # sum of H squares, halved by the root; division, root, mean, eps and two products
    err = np.abs(want) * (H * 2.0 ** -24 + 8 * 2.0 ** -24)
    check_rows(y8, ys, want, err)
    off = np.abs(f64(bits(y)) - want)
    assert (off <= np.abs(want) * 2.0 ** -8 + 2 * err + 2.0 ** -134).all()


@pytest.mark.parametrize("H", [16, 64, 128, 144, 512, 528, 1024, 2048, 2064, 4096, 7168, 8192, 8208, 16384, 16400])
def test_norm_widths(H):
    rng = np.random.default_rng(H)
    for N in (1, 5, 67):
        print(f"[case] norm N={N} H={H}", flush=True)
        x = bf16_of(rng.standard_normal((N, H)))
        res = bf16_of(rng.standard_normal((N, H)) * 4)
        w = bf16_of(1 + 0.2 * rng.standard_normal(H))
        check_norm(x, res, w, 1e-6)
        check_norm(x, res, w, 1e-6, inplace=True)
        check_norm(x, None, w, 1e-5)


def test_norm_widest_row():
    rng = np.random.default_rng(0)
    print("[case] norm N=3 H=65536", flush=True)
    check_norm(bf16_of(rng.standard_normal((3, 65536))), bf16_of(rng.standard_normal((3, 65536))),
               bf16_of(np.ones(65536)), 1e-6)


def test_norm_many_rows():
    """More rows than one grid holds of the largest workgroups' worth of rows."""
    rng = np.random.default_rng(1)
    print("[case] norm N=70001 H=64", flush=True)
    x = bf16_of(rng.standard_normal((70001, 64)))
    check_norm(x, x[::-1].copy(), bf16_of(np.ones(64)), 1e-6)


def test_norm_zero_rows_and_blocks():
    rng = np.random.default_rng(2)
    x = bf16_of(rng.standard_normal((4, 512)))
    x[0] = 0
    x[1, 128:256] = 0
    w = bf16_of(np.ones(512))
    check_norm(x, None, w, 1e-6)
    # cancelling residual: r is 0, every scale 1
    out, y, y8, ys = run_norm(x, x ^ np.uint16(0x8000), w, 1e-6)
    assert (f64(bits(out)) == 0).all() and (y8 & 0x7F == 0).all() and (ys == 127).all()


def test_norm_magnitudes():
    """Rows of tiny and of large values, whose squares still fit fp32; scales at the border 448 * 2^e."""
    rng = np.random.default_rng(3)
    w = bf16_of(2.0 ** rng.integers(-60, 60, 256))
    x = np.stack([rng.standard_normal(256) * 2.0 ** k for k in (-55, -20, 0, 20, 55)])
    check_norm(bf16_of(x), None, w, 0.0)


def test_norm_non_finite():
    """A NaN makes its row NaN; an infinite value is NaN, and 0 elsewhere in its row; other rows are as ever."""
    rng = np.random.default_rng(4)
    x = f64(bf16_of(rng.standard_normal((5, 256))))
    x[1, 7] = np.nan
    x[3, 200] = np.inf
    w = bf16_of(np.ones(256))
    _, y, y8, ys = run_norm(bf16_of(x), None, w, 1e-6)
    assert (ys[1, :2] == 255).all() and (y8[1] == 0x7F).all() and np.isnan(f64(bits(y))[1]).all()
    assert ys[3, 1] == 255 and (y8[3, 128:] == 0x7F).all()
    assert ys[3, 0] == 127 and (y8[3, :128] & 0x7F == 0).all()
    _, _, c8, cs = run_norm(bf16_of(x[[0, 2, 4]]), None, w, 1e-6)
    np.testing.assert_array_equal(y8[[0, 2, 4]], c8)
    np.testing.assert_array_equal(ys[[0, 2, 4]], cs)


def test_norm_without_bf16_output_and_empty():
    rng = np.random.default_rng(5)
    x, w = bf16_of(rng.standard_normal((9, 256))), bf16_of(np.ones(256))
    a, b = run_norm(x, None, w, 1e-6), run_norm(x, None, w, 1e-6, want_y=False)
    np.testing.assert_array_equal(a[2], b[2])
    np.testing.assert_array_equal(a[3], b[3])
    run_norm(x[:0], x[:0], w, 1e-6)


# ---------------------------------------------------------------------------
# dispatch
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("R,E,S,K,H", [(1, 4, 1, 1, 16), (4, 16, 13, 2, 80), (8, 32, 33, 8, 1040), (2, 12, 50, 12, 528),
                                       (2, 8, 31, 3, 2048), (1, 8, 9, 5, 9216)])
def test_dispatch_copies_rows(R, E, S, K, H):
    print(f"[case] dispatch R={R} E={E} S={S} K={K} H={H}", flush=True)
    w = synth.Workload("d", R, E, S, K, H, "zipf", alpha=1.2)
    topk, _ = synth.routing(w, 0)
    _, _, _, slot_of, _ = oracle_plan(w, topk)
    rng = np.random.default_rng(0)
    x8 = rng.integers(0, 256, (w.N, H), dtype=np.uint8)
    xs = rng.integers(0, 256, (w.N, scale_bytes(H)), dtype=np.uint8)
    slots = slot_of.copy()
    slots[::7] = -1  # entries a planner refused, and one past the end
    slots[1::11] = w.NK
    buf8 = torch.full((w.NK, H), 0xA5, dtype=torch.uint8, device="cuda")
    bufs = torch.full((w.NK, scale_bytes(H)), 0xA5, dtype=torch.uint8, device="cuda")
    mx.moonep_dispatch_quant(shape_of(w), to_dev(x8), to_dev(xs), to_dev(slots), buf8, bufs)
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < w.NK)
    want8, wants = np.full((w.NK, H), 0xA5, np.uint8), np.full((w.NK, scale_bytes(H)), 0xA5, np.uint8)
    want8[slots[ok]] = x8[np.arange(w.NK)[ok] // K]
    wants[slots[ok]] = xs[np.arange(w.NK)[ok] // K]
    np.testing.assert_array_equal(host(buf8), want8)
    np.testing.assert_array_equal(host(bufs), wants)


# ---------------------------------------------------------------------------
# weights
# ---------------------------------------------------------------------------

def quantise_matrix(m):
    """Codes and block scales of an [out, in] matrix of bf16 values, by definition."""
    out, inp = m.shape
    ob, ib = -(-out // 128), -(-inp // 128)
    s = np.full((ob, scale_bytes(inp)), 127, np.uint8)
    p = np.zeros((ob * 128, ib * 128))
    p[:out, :inp] = np.abs(m)
    s[:, :ib] = scale_of(p.reshape(ob, 128, ib, 128).max((1, 3)))
    per = np.repeat(expand(s, inp), 128, axis=0)[:out]
    v = torch.from_numpy((m / per).astype(np.float32)).to(torch.float8_e4m3fn)
    return v.view(torch.uint8).numpy(), s


@pytest.mark.parametrize("E,out,inp", [(1, 1, 16), (3, 128, 128), (2, 130, 144), (4, 208, 336), (2, 257, 2048), (1, 96, 4112)])
def test_weights_exact(E, out, inp):
    print(f"[case] weights E={E} out={out} in={inp}", flush=True)
    rng = np.random.default_rng(out)
    n, nscale = out * inp, -(-out // 128) * scale_bytes(inp)
    w_off, w_stride = 24, 24 + n + 16
    scale_off = 16
    code_off = scale_off + nscale + (-(scale_off + nscale)) % 16 + 32
    stride = code_off + n + 48
    m = bf16_of(rng.standard_normal((E, w_stride)) * 2.0 ** rng.integers(-12, 12, (E, w_stride)))
    m[0, w_off:w_off + 16] = 0
    w8 = torch.full((E, stride), 0x5A, dtype=torch.uint8, device="cuda")
    mx.moonep_quant_weights(mx.Shape(1, E, 0, 1, 16), inp, out, bf16_dev(m), w_stride, w_off, w8, stride, code_off,
                            scale_off)
    torch.cuda.synchronize()
    got = host(w8)
    want = np.full((E, stride), 0x5A, np.uint8)
    for e in range(E):
        c, s = quantise_matrix(f64(m[e, w_off:w_off + n]).reshape(out, inp))
        want[e, code_off:code_off + n] = c.reshape(-1)
        want[e, scale_off:scale_off + nscale] = s.reshape(-1)
    np.testing.assert_array_equal(got, want)


def test_weights_border_and_non_finite():
    """Largest magnitudes at the border of two scales, ties between codes, and blocks that hold an infinity or a NaN."""
    m = np.zeros((128, 512))
    m[0, 0], m[0, 1] = 448.0, 449.0 - 1.0
    m[0, 128], m[1, 129] = 450.0, 17.0          # 450 > 448: the next scale; 17 / 2 = 8.5 is a tie
    m[5, 256] = np.inf
    m[9, 400] = np.nan
    b = bf16_of(m)
    w8 = torch.zeros((1, 128 * 512 + 16), dtype=torch.uint8, device="cuda")
    mx.moonep_quant_weights(mx.Shape(1, 1, 0, 1, 16), 512, 128, bf16_dev(b.reshape(1, -1)), 128 * 512, 0, w8,
                            128 * 512 + 16, 0, 128 * 512)
    torch.cuda.synchronize()
    g = host(w8)[0]
    codes, s = g[:128 * 512].reshape(128, 512), g[128 * 512:128 * 512 + 4]
    assert s.tolist() == [127, 128, 255, 255]
    assert (codes[:, 256:] == 0x7F).all()
    want, _ = quantise_matrix(f64(b)[:, :256])
    np.testing.assert_array_equal(codes[:, :256], want)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

PRODUCTS = [
    # workload, in, out, B
    (synth.Workload("one_token", 1, 8, 1, 2, 16, "zipf"), 128, 128, 0),
    (synth.Workload("decode", 8, 64, 4, 8, 16, "zipf", alpha=1.0), 512, 384, 3),
    (synth.Workload("odd", 4, 16, 27, 3, 16, "zipf", alpha=1.5), 336, 208, 1),
    (synth.Workload("narrow", 2, 4, 40, 2, 16, "zipf", alpha=1.0), 16, 16, 1),
    (synth.Workload("skewed", 4, 16, 200, 4, 16, "zipf", alpha=2.5), 640, 272, 2),
    (synth.Workload("overflow", 8, 32, 128, 4, 16, "zipf", alpha=2.0), 1104, 400, 0),
    (synth.Workload("to_one_rank", 8, 32, 96, 4, 16, "fixed", gates="uniform"), 256, 144, 4),
    (synth.Workload("tall", 1, 2, 700, 1, 16, "zipf"), 1408, 528, 0),
    (synth.Workload("most_experts", 512, 1024, 4, 2, 16, "zipf", alpha=1.2), 64, 48, 1),
]


def product_setup(w, B, seed=0):
    topk, _ = synth.routing(w, seed)
    _, _, pl, _, _ = oracle_plan(w, topk)
    b = mx.allocate(shape_of(w))
    mx.plan_step(b, to_dev(topk))
    ws = torch.empty(w.E + w.R, dtype=torch.int32, device="cuda")
    mx.moonep_weight_slots(b.shape, b.plan, B, ws)
    o_ws = oracle.weight_slots(w.R, w.E, B, pl)
    # (first row, rows, pooled, weight row) of every segment
    C, L = w.C, w.E // w.R
    segs = [((e // L) * C + int(pl.home_row_off[e]), int(pl.keep[e]), False, e) for e in range(w.E)]
    for j in range(pl.n_rep):
        q = int(o_ws[j])
        segs.append((int(pl.rep_host[j]) * C + int(pl.rep_row_off[j]), int(pl.rep_count[j]), q >= 0,
                     q if q >= 0 else int(pl.rep_expert[j])))
    return b, ws, [s for s in segs if s[1]]


def weight_rows(rng, rows, mats, integers, finite=True):
    """[rows, stride] bytes with codes and scales of every matrix, their windows.
    Without `finite` the few normal values past 448 become NaN codes."""
    at, wins = 32, []
    for out, inp in mats:
        scale, at = at, at + -(-out // 128) * scale_bytes(inp)
        at += -at % 16 + 16
        code, at = at, at + out * inp
        wins.append((code, scale))
        at += -at % 16
    w = rng.integers(0, 256, (rows, at + 16), dtype=np.uint8)
    for (out, inp), (code, scale) in zip(mats, wins):
        n = -(-out // 128) * scale_bytes(inp)
        if integers:
            v = torch.from_numpy(rng.integers(-4, 5, (rows, out * inp)).astype(np.float32))
            w[:, code:code + out * inp] = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            w[:, scale:scale + n] = rng.integers(126, 129, (rows, n))
        else:
            v = torch.from_numpy((rng.standard_normal((rows, out * inp)) * 100).astype(np.float32))
            v = v.clamp(-448, 448) if finite else v
            w[:, code:code + out * inp] = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            w[:, scale:scale + n] = rng.integers(112, 120, (rows, n))
    return w, wins


def x_rows(rng, rows, cols, integers):
    if integers:
        v = torch.from_numpy(rng.integers(-4, 5, (rows, cols)).astype(np.float32))
        return (v.to(torch.float8_e4m3fn).view(torch.uint8).numpy(),
                rng.integers(126, 129, (rows, scale_bytes(cols)), dtype=np.uint8))
    return quantise(rng.standard_normal((rows, cols)).astype(np.float32).astype(np.float64))


def reference(segs, x8, xs, w_home, pool, mats, wins):
    """Every product [rows, out] in fp64 and the sum of its terms' magnitudes."""
    got = []
    for (out, inp), (code, scale) in zip(mats, wins):
        y = np.zeros((x8.shape[0], out))
        a = np.zeros((x8.shape[0], out))
        for row0, n, pooled, wrow in segs:
            wr = (pool if pooled else w_home)[wrow]
            wv = weight_values(wr[code:code + out * inp].reshape(out, inp),
                               wr[scale:scale + -(-out // 128) * scale_bytes(inp)].reshape(-1, scale_bytes(inp)))
            xv = values(x8[row0:row0 + n], xs[row0:row0 + n])
            y[row0:row0 + n] = xv @ wv.T
            a[row0:row0 + n] = np.abs(xv) @ np.abs(wv).T
        got.append((y, a))
    return got


def run_gemm(w, b, ws, B, inp, out, x8, xs, w_home, pool, win):
    y = torch.empty((w.NK, out), dtype=torch.bfloat16, device="cuda")
    y.view(torch.int16).fill_(-1)
    mx.moonep_expert_gemm_quant(b.shape, b.plan, ws, B, inp, out, codes_dev(x8), to_dev(xs), to_dev(w_home),
                                to_dev(pool), w_home.shape[1], *win, y)
    torch.cuda.synchronize()
    return y


def run_glu(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins):
    h8 = torch.full((w.NK, out), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((w.NK, scale_bytes(out)), 0x55, dtype=torch.uint8, device="cuda")
    mx.moonep_expert_glu_quant(b.shape, b.plan, ws, B, inp, out, codes_dev(x8), to_dev(xs), to_dev(w_home),
                               to_dev(pool), w_home.shape[1], *wins[0], *wins[1], h8, hs)
    torch.cuda.synchronize()
    return host(h8), host(hs)


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: c[0].name)
def test_gemm_integers_bit_exact(case):
    """Small integers times powers of two: every partial sum is exact in fp32, so
    the outputs are the one rounding to bf16 of the true sums."""
    w, inp, out, B = case
    print(f"[case] gemm {w.name} in={inp} out={out} B={B}", flush=True)
    rng = np.random.default_rng(1)
    b, ws, segs = product_setup(w, B)
    w_home, wins = weight_rows(rng, w.E, [(out, inp)], True)
    pool, _ = weight_rows(rng, w.R * B, [(out, inp)], True)
    x8, xs = x_rows(rng, w.NK, inp, True)
    y = run_gemm(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins[0])
    (want, _), = reference(segs, x8, xs, w_home, pool, [(out, inp)], wins)
    np.testing.assert_array_equal(bits(y), bf16_of(want))


@pytest.mark.parametrize("case", PRODUCTS[:-1], ids=lambda c: c[0].name)
def test_gemm_real_within_bound(case):
    w, inp, out, B = case
    print(f"[case] gemm real {w.name}", flush=True)
    rng = np.random.default_rng(2)
    b, ws, segs = product_setup(w, B)
    w_home, wins = weight_rows(rng, w.E, [(out, inp)], False, finite=False)
    pool, _ = weight_rows(rng, w.R * B, [(out, inp)], False, finite=False)
    x8, xs = x_rows(rng, w.NK, inp, False)
    y = f64(bits(run_gemm(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins[0])))
    (want, a), = reference(segs, x8, xs, w_home, pool, [(out, inp)], wins)
    # the columns of NaN codes, and no others
    np.testing.assert_array_equal(np.isnan(y), np.isnan(want))
    ok = ~np.isnan(want)
    assert ok.mean() > 0.9
    off, allowed = np.abs(y - want), np.abs(want) * 2.0 ** -8 + 2 * inp * 2.0 ** -23 * a + 2.0 ** -134
    assert (off[ok] <= allowed[ok]).all(), f"{(off[ok] / allowed[ok]).max()} of what is allowed"


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: c[0].name)
def test_glu_within_bound(case):
    w, inp, out, B = case
    print(f"[case] glu {w.name}", flush=True)
    rng = np.random.default_rng(3)
    b, ws, segs = product_setup(w, B)
    mats = [(out, inp), (out, inp)]
    w_home, wins = weight_rows(rng, w.E, mats, False)
    pool, _ = weight_rows(rng, w.R * B, mats, False)
    x8, xs = x_rows(rng, w.NK, inp, False)
    h8, hs = run_glu(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins)
    (g, ga), (u, ua) = reference(segs, x8, xs, w_home, pool, mats, wins)
    silu = g / (1 + np.exp(-g))
    # the slope of silu is below 1.1; its exponential is good to 2^-22 + |g| 2^-23, and the rest to 2^-21
    dg, du = inp * 2.0 ** -23 * ga, inp * 2.0 ** -23 * ua
    h = silu * u
    err = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + np.abs(h) * (np.abs(g) + 4) * 2.0 ** -22
    check_rows(h8, hs, h, err)


# Hundreds of rows an expert, so the tile of 256 rows: fewer k-steps than the ring has stages, all items halves of
# a tile, and one or two rounds of whole tiles before a round of halves.
TALL = [
    (synth.Workload("one_step", 1, 2, 1500, 1, 16, "zipf"), 16, 48, 0),
    (synth.Workload("two_steps", 2, 4, 700, 2, 16, "zipf", alpha=1.0), 144, 272, 1),
    (synth.Workload("half_round", 1, 4, 4400, 1, 16, "zipf", alpha=0.5), 32, 4096, 0),
]


@pytest.mark.parametrize("case", TALL, ids=lambda c: c[0].name)
def test_gemm_large_tiles(case):
    w, inp, out, B = case
    print(f"[case] gemm {w.name} in={inp} out={out} B={B}", flush=True)
    rng = np.random.default_rng(6)
    b, ws, segs = product_setup(w, B)
    w_home, wins = weight_rows(rng, w.E, [(out, inp)], True)
    pool, _ = weight_rows(rng, w.R * B, [(out, inp)], True)
    x8, xs = x_rows(rng, w.NK, inp, True)
    y = run_gemm(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins[0])
    (want, _), = reference(segs, x8, xs, w_home, pool, [(out, inp)], wins)
    np.testing.assert_array_equal(bits(y), bf16_of(want))


@pytest.mark.parametrize("case", TALL, ids=lambda c: c[0].name)
def test_glu_large_tiles(case):
    w, inp, out, B = case
    print(f"[case] glu {w.name}", flush=True)
    rng = np.random.default_rng(7)
    b, ws, segs = product_setup(w, B)
    mats = [(out, inp), (out, inp)]
    w_home, wins = weight_rows(rng, w.E, mats, False)
    pool, _ = weight_rows(rng, w.R * B, mats, False)
    x8, xs = x_rows(rng, w.NK, inp, False)
    h8, hs = run_glu(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins)
    (g, ga), (u, ua) = reference(segs, x8, xs, w_home, pool, mats, wins)
    silu = g / (1 + np.exp(-g))
    # fp32 sums, and 2^-16 of the magnitudes for what the matrix instruction drops inside itself
    dg, du = (inp * 2.0 ** -23 + 2.0 ** -16) * ga, (inp * 2.0 ** -23 + 2.0 ** -16) * ua
    h = silu * u
    err = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + np.abs(h) * (np.abs(g) + 4) * 2.0 ** -22
    check_rows(h8, hs, h, err)


def test_products_of_non_finite_rows():
    """A NaN code or scale in a row makes that row's outputs NaN and no other's."""
    w, inp, out, B = PRODUCTS[4]
    rng = np.random.default_rng(4)
    b, ws, segs = product_setup(w, B)
    mats = [(out, inp), (out, inp)]
    w_home, wins = weight_rows(rng, w.E, mats, False)
    pool, _ = weight_rows(rng, w.R * B, mats, False)
    x8, xs = x_rows(rng, w.NK, inp, False)
    base = bits(run_gemm(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins[0]))
    base8, bases = run_glu(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins)
    x8[3, 5], xs[17, 1] = 0x7F, 255
    y = bits(run_gemm(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins[0]))
    h8, hs = run_glu(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins)
    bad = np.zeros(w.NK, bool)
    bad[[3, 17]] = True
    assert np.isnan(f64(y[bad])).all() and (h8[bad] == 0x7F).all()
    assert (hs[bad][:, :-(-out // 128)] == 255).all()
    np.testing.assert_array_equal(y[~bad], base[~bad])
    np.testing.assert_array_equal(h8[~bad], base8[~bad])
    np.testing.assert_array_equal(hs[~bad], bases[~bad])


def test_products_empty():
    w = synth.Workload("none", 4, 16, 0, 2, 16, "balanced")
    b = mx.allocate(shape_of(w))
    ws = torch.full((w.E + w.R,), -1, dtype=torch.int32, device="cuda")
    row = torch.zeros((w.E, 128 * 128 + 16), dtype=torch.uint8, device="cuda")
    e8 = torch.empty((0, 128), dtype=torch.uint8, device="cuda")
    es = torch.empty((0, 4), dtype=torch.uint8, device="cuda")
    mx.moonep_expert_gemm_quant(b.shape, b.plan, ws, 0, 128, 128, e8, es, row, None, row.shape[1], 0, 128 * 128,
                                torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()


def test_products_full_size():
    """The sweep shape's gate and up, and down, on sampled rows (the tile the
    large calls take, every XCD and rank at work)."""
    w = synth.sweep_workload(1.0, seed=0)
    F, B = synth.SWEEP_FFN, w.E // w.R
    print("[case] sweep products", flush=True)
    b, ws, segs = product_setup(w, B)
    rng = np.random.default_rng(5)
    g = torch.Generator(device="cuda").manual_seed(5)

    def draw(rows, cols):
        v = torch.randn((rows, cols), generator=g, device="cuda") * 100
        return v.clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales(rows, n, lo, hi):
        return torch.randint(lo, hi, (rows, n), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)

    for kind, inp, out in (("glu", w.H, F), ("gemm", F, w.H)):
        mats = [(out, inp)] * (2 if kind == "glu" else 1)
        n, ns = out * inp, out // 128 * scale_bytes(inp)
        wins = [(m * n, len(mats) * n + m * ns) for m in range(len(mats))]
        stride = len(mats) * (n + ns)
        w_home = torch.empty((w.E, stride), dtype=torch.uint8, device="cuda")
        w_home[:, :len(mats) * n] = draw(w.E, len(mats) * n).view(torch.uint8)
        w_home[:, len(mats) * n:] = scales(w.E, len(mats) * ns, 112, 118)
        pool = torch.zeros((w.R * B, stride), dtype=torch.uint8, device="cuda")
        mx.moonep_prefetch_weights(b.shape, b.plan, ws, B, stride, w_home, pool)
        x8, xs = draw(w.NK, inp), scales(w.NK, scale_bytes(inp), 118, 122)
        rows = np.unique(np.concatenate([rng.integers(0, w.NK, 48), [0, w.NK - 1],
                                         [s[0] + s[1] - 1 for s in segs[::7]]]))
        rd = torch.from_numpy(rows).cuda()
        if kind == "glu":
            h8 = torch.full((w.NK, out), 0x55, dtype=torch.uint8, device="cuda")
            hs = torch.full((w.NK, scale_bytes(out)), 0x55, dtype=torch.uint8, device="cuda")
            mx.moonep_expert_glu_quant(b.shape, b.plan, ws, B, inp, out, x8, xs, w_home, pool, stride, *wins[0],
                                       *wins[1], h8, hs)
        else:
            y = torch.full((w.NK, out), float("nan"), dtype=torch.bfloat16, device="cuda")
            mx.moonep_expert_gemm_quant(b.shape, b.plan, ws, B, inp, out, x8, xs, w_home, pool, stride, *wins[0], y)
        torch.cuda.synchronize()
        sx8, sxs = host(x8[rd]), host(xs[rd])
        outs = [[np.zeros((rows.size, out)), np.zeros((rows.size, out))] for _ in mats]
        for row0, cnt, pooled, wrow in segs:
            sel = np.nonzero((rows >= row0) & (rows < row0 + cnt))[0]
            if not sel.size:
                continue
            wr = host((pool if pooled else w_home)[wrow])
            for o, (code, scale) in zip(outs, wins):
                wv = weight_values(wr[code:code + n].reshape(out, inp), wr[scale:scale + ns].reshape(-1, scale_bytes(inp)))
                xv = values(sx8[sel], sxs[sel])
                o[0][sel], o[1][sel] = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        if kind == "glu":
            (gv, ga), (uv, ua) = outs
            silu = gv / (1 + np.exp(-gv))
            dg, du = inp * 2.0 ** -23 * ga, inp * 2.0 ** -23 * ua
            h = silu * uv
            err = 1.1 * dg * np.abs(uv) + (np.abs(silu) + 1.1 * dg) * du + np.abs(h) * (np.abs(gv) + 4) * 2.0 ** -22
            check_rows(host(h8[rd]), host(hs[rd]), h, err)
        else:
            (want, a), = outs
            assert not torch.isnan(y).any()
            off = np.abs(f64(bits(y[rd])) - want)
            assert (off <= np.abs(want) * 2.0 ** -8 + 2 * inp * 2.0 ** -23 * a).all()


def test_far_rows():
    """Rows more than 2^32 bytes into their arrays: norm, dispatch and a product, on the first, some middle and the
    last rows."""
    g = torch.Generator(device="cuda").manual_seed(7)
    N, K, H, F = (1 << 20) + 5, 2, 2064, 16
    s = mx.Shape(1, 2, N, K, H)
    rows = torch.tensor([0, 1, N // 2, N - 2, N - 1], device="cuda")
    print("[case] far rows", flush=True)
    x = torch.randn((N, H), generator=g, device="cuda", dtype=torch.bfloat16)      # 4.3 GB
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y8 = torch.zeros((N, H), dtype=torch.uint8, device="cuda")
    ys = torch.zeros((N, scale_bytes(H)), dtype=torch.uint8, device="cuda")
    mx.moonep_rmsnorm_quant(s, x, None, w, 1e-6, None, None, y8, ys)
    v = x[rows].double().cpu().numpy()
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
    check_rows(host(y8[rows]), host(ys[rows]), want, np.abs(want) * (H + 8) * 2.0 ** -24)
    del x
    # every token to both experts, in either order
    topk = torch.stack([torch.arange(N, device="cuda") % 2, (torch.arange(N, device="cuda") + 1) % 2], 1).int().reshape(-1)
    b = mx.allocate(mx.Shape(1, 2, N, K, 8))
    mx.plan_step(b, topk.contiguous())
    buf8 = torch.zeros((N * K, H), dtype=torch.uint8, device="cuda")               # 4.3 GB
    bufs = torch.zeros((N * K, scale_bytes(H)), dtype=torch.uint8, device="cuda")
    mx.moonep_dispatch_quant(s, y8, ys, b.slot_of, buf8, bufs)
    assert int(b.slot_of.max()) == N * K - 1
    for k in range(K):
        at = b.slot_of.view(N, K)[rows, k].long()
        assert torch.equal(buf8[at], y8[rows]) and torch.equal(bufs[at], ys[rows])
    rng = np.random.default_rng(7)
    w_home, wins = weight_rows(rng, 2, [(F, H)], False)
    ws = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    y = torch.full((N * K, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    mx.moonep_expert_gemm_quant(s, b.plan, ws, 0, H, F, buf8, bufs, to_dev(w_home), None, w_home.shape[1], *wins[0], y)
    torch.cuda.synchronize()
    assert not torch.isnan(y).any()
    code, scale = wins[0]
    for k in range(K):
        at = b.slot_of.view(N, K)[rows, k].long()
        got = f64(bits(y[at]))
        xv = values(host(buf8[at]), host(bufs[at]))
        for i, e in enumerate(topk.view(N, K)[rows, k].cpu().tolist()):
            wv = weight_values(w_home[e, code:code + F * H].reshape(F, H),
                               w_home[e, scale:scale + scale_bytes(H)].reshape(1, -1))
            o, a = wv @ xv[i], np.abs(wv) @ np.abs(xv[i])
            assert (np.abs(got[i] - o) <= np.abs(o) * 2.0 ** -8 + 2 * H * 2.0 ** -23 * a).all()
