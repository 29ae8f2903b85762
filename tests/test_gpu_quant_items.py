"""The 8-bit kernels past their first item: more items than workgroups, so that each workgroup's rings of loads and
scales run on into the next item under the epilogue (products), its next rows are on their way and its LDS buffers
change over (weights), and its grid strides over the rows (norm, dispatch).  Bounds and helpers as in
test_gpu_quant.py."""
import numpy as np
import pytest
import torch

import load_balancing_amd as mx
import synth
from gpu_harness import bf16_dev, bits, to_dev
from quant_ref import check_rows, host, scale_bytes
from test_gpu_quant import (bf16_of, f64, product_setup, quantise_matrix, reference, run_gemm, run_glu, run_norm,
                            weight_rows, x_rows)

pytestmark = pytest.mark.gpu


def items(segs, rows, cols, out):
    """Tiles of `rows` rows in the segments, times column blocks."""
    return sum(-(-n // rows) for _, n, _, _ in segs) * -(-out // cols)


def two_rounds(n):
    """Some workgroups take a third item at least: one workgroup per compute unit, two at most."""
    return n > 2 * torch.cuda.get_device_properties(0).multi_processor_count


def work(rows, seed=0):
    """64 experts on 8 ranks with about `rows` rows each."""
    return synth.Workload(f"mean{rows}", 8, 64, rows, 8, 16, "zipf", alpha=0.6)


# mean rows of an expert, rows and columns of its tile, in (8 to 16 k-steps: more than any ring, and than a dword of
# scales has blocks; one with part of a k-step), out
GEMM = [(8, 32, 128, 1040, 2048), (20, 32, 128, 2048, 1424), (96, 128, 128, 1040, 1424), (60, 128, 128, 2048, 2048),
        (200, 256, 256, 1040, 2320)]
GLU = [(8, 32, 128, 1040, 1424), (12, 32, 128, 2048, 1152), (40, 64, 128, 1040, 1424), (80, 64, 128, 2048, 1152),
       (200, 256, 128, 1040, 1168)]


@pytest.mark.parametrize("mean,bm,bn,inp,out", GEMM)
def test_gemm_next_items_bit_exact(mean, bm, bn, inp, out):
    print(f"[case] gemm items mean={mean} in={inp} out={out}", flush=True)
    rng = np.random.default_rng(31)
    w, B = work(mean), 2
    b, ws, segs = product_setup(w, B)
    assert two_rounds(items(segs, bm, bn, out))
    w_home, wins = weight_rows(rng, w.E, [(out, inp)], True)
    pool, _ = weight_rows(rng, w.R * B, [(out, inp)], True)
    x8, xs = x_rows(rng, w.NK, inp, True)
    y = run_gemm(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins[0])
    (want, _), = reference(segs, x8, xs, w_home, pool, [(out, inp)], wins)
    np.testing.assert_array_equal(bits(y), bf16_of(want))


@pytest.mark.parametrize("mean,bm,bn,inp,out", GLU)
def test_glu_next_items(mean, bm, bn, inp, out):
    print(f"[case] glu items mean={mean} in={inp} out={out}", flush=True)
    rng = np.random.default_rng(32)
    w, B = work(mean), 2
    b, ws, segs = product_setup(w, B)
    assert two_rounds(items(segs, bm, bn, out))
    mats = [(out, inp), (out, inp)]
    w_home, wins = weight_rows(rng, w.E, mats, False)
    pool, _ = weight_rows(rng, w.R * B, mats, False)
    x8, xs = x_rows(rng, w.NK, inp, False)
    h8, hs = run_glu(w, b, ws, B, inp, out, x8, xs, w_home, pool, wins)
    (g, ga), (u, ua) = reference(segs, x8, xs, w_home, pool, mats, wins)
    silu = g / (1 + np.exp(-g))
    dg, du = inp * 2.0 ** -23 * ga, inp * 2.0 ** -23 * ua
    h = silu * u
    err = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + np.abs(h) * (np.abs(g) + 4) * 2.0 ** -22
    check_rows(h8, hs, h, err)


def test_weights_next_items():
    """1760 items (128 x 512 values each, ragged in both) for at most 512 workgroups."""
    E, out, inp = 40, 1300, 1552
    print(f"[case] weights items E={E} out={out} in={inp}", flush=True)
    rng = np.random.default_rng(33)
    n, nscale = out * inp, -(-out // 128) * scale_bytes(inp)
    scale_off = n + (-n) % 16
    stride = scale_off + nscale + (-(scale_off + nscale)) % 16
    m = bf16_of(rng.standard_normal((E, n), dtype=np.float32) * np.exp2(rng.integers(-9, 9, (E, 1))).astype(np.float32))
    w8 = torch.full((E, stride), 0x5A, dtype=torch.uint8, device="cuda")
    mx.moonep_quant_weights(mx.Shape(1, E, 0, 1, 16), inp, out, bf16_dev(m), n, 0, w8, stride, 0, scale_off)
    torch.cuda.synchronize()
    got = host(w8)
    for e in range(E):
        c, s = quantise_matrix(f64(m[e]).reshape(out, inp))
        np.testing.assert_array_equal(got[e, :n].reshape(out, inp), c, err_msg=f"codes of expert {e}")
        np.testing.assert_array_equal(got[e, scale_off:scale_off + nscale].reshape(s.shape), s)


def test_norm_and_dispatch_rows_past_one_grid():
    """2^22 rows are what one grid of the narrow norm, and of a dispatch of narrow rows, holds: some more."""
    N, H = (1 << 22) + 4099, 16
    print(f"[case] norm and dispatch N={N} H={H}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(34)
    x = torch.randn((N, H), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y8 = torch.full((N, H), 0x55, dtype=torch.uint8, device="cuda")
    ys = torch.full((N, 4), 0x55, dtype=torch.uint8, device="cuda")
    s = mx.Shape(1, 1, N, 1, H)
    mx.moonep_rmsnorm_quant(s, x, None, w, 1e-6, None, None, y8, ys)
    # the rows around and past 2^22, and some of the others; 8-bit rows of all others in their place
    some = torch.cat([torch.randint(0, N, (4000,), generator=g, device="cuda"),
                      torch.arange((1 << 22) - 50, N, device="cuda")])
    v = x[some].double().cpu().numpy()
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6)
    check_rows(host(y8[some]), host(ys[some]), want, np.abs(want) * (H + 8) * 2.0 ** -24)
    near = y8.view(torch.float8_e4m3fn).float() * ys.view(torch.float8_e8m0fnu).float()[:, :1]
    v = x.float()
    v *= torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    assert ((near - v).abs() <= v.abs() * 2.0 ** -3 + 2.0 ** -8).all()  # twice a half step: which row, not which code
    slot = torch.arange(N, device="cuda", dtype=torch.int32).flip(0).contiguous()
    buf8 = torch.full((N, H), 0xA5, dtype=torch.uint8, device="cuda")
    bufs = torch.full((N, 4), 0xA5, dtype=torch.uint8, device="cuda")
    mx.moonep_dispatch_quant(s, y8, ys, slot, buf8, bufs)
    assert torch.equal(buf8, y8.flip(0)) and torch.equal(bufs, ys.flip(0))


def test_norm_rows_without_squares():
    """With eps = 0, rows of zeros or of values of 2^-80 have no norm in fp32: codes and scales say so, the rows beside
    them are as ever.  Any eps gives them one."""
    x = np.ones((4, 256))
    x[1], x[2] = 0, 2.0 ** -80
    w = bf16_of(np.ones(256))
    _, y, y8, ys = run_norm(bf16_of(x), None, w, 0.0)
    assert (ys[1:3, :2] == 255).all() and (y8[1:3] == 0x7F).all() and not np.isfinite(f64(bits(y))[1:3]).any()
    assert (f64(bits(y))[[0, 3]] == 1).all()
    _, y, y8, ys = run_norm(bf16_of(x), None, w, 1e-30)
    assert (f64(bits(y))[1] == 0).all() and (ys[1] == 127).all()
    want = 2.0 ** -80 / np.sqrt(1e-30)
    assert (np.abs(f64(bits(y))[2] - want) <= want * 2.0 ** -7).all()
