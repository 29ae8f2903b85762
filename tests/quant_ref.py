"""References in 64 bits for the 8-bit rows, and the checks of a quantised
output against real values, for the tests of the 8-bit path.

A scale is the least power of two that brings its block's largest magnitude to
at most 448; a code is at most half a step off: 2^-4 of the value relative
(three bits after the leading one), and never under 2^-10 of the scale (the step
of the smallest codes is 2^-9)."""
import numpy as np
import torch

BLOCK = 128
CODE_BYTES = np.arange(256, dtype=np.uint8)
CODE_VALUES = torch.from_numpy(CODE_BYTES.copy()).view(torch.float8_e4m3fn).double().numpy()


def scale_bytes(cols):
    return 4 * -(-cols // (4 * BLOCK))


def host(t):
    """uint8 array of a tensor of codes or scales."""
    return t.contiguous().view(torch.uint8).cpu().numpy()


def scale_values(s):
    v = np.ldexp(1.0, s.astype(np.int64) - 127)
    return np.where(s == 255, np.nan, v)


def expand(s, cols):
    """[rows, scale bytes] -> [rows, cols] scales."""
    return np.repeat(scale_values(s), BLOCK, axis=1)[:, :cols]


def values(codes, s):
    return CODE_VALUES[codes] * expand(s, codes.shape[1])


def weight_values(codes, s):
    """[out, in] codes and [ceil(out / 128), scale bytes] scales of 128 x 128 blocks."""
    return CODE_VALUES[codes] * np.repeat(expand(s, codes.shape[1]), BLOCK, axis=0)[:codes.shape[0]]


def block_amax(y):
    rows, cols = y.shape
    nb = -(-cols // BLOCK)
    p = np.zeros((rows, nb * BLOCK))
    p[:, :cols] = np.abs(y)
    return p.reshape(rows, nb, BLOCK).max(2)


def scale_of(amax):
    """E8M0 byte of a finite block's largest magnitude."""
    m, e = np.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    b = np.where(m <= 0.875, e - 9, e - 8) + 127
    return np.where(amax == 0, 127, np.maximum(b, 1))


def quantise(y):
    """Codes and padded scales of [rows, cols] values that are exact in fp32."""
    rows, cols = y.shape
    nb = -(-cols // BLOCK)
    s = np.full((rows, scale_bytes(cols)), 127, np.uint8)
    s[:, :nb] = scale_of(block_amax(y))
    v = (y / expand(s, cols)).astype(np.float32)
    return torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), s


def check_rows(codes, s, y, err):
    """8-bit rows of y, known to within err (elementwise, from the arithmetic
    before the quantisation)."""
    rows, cols = y.shape
    nb = -(-cols // BLOCK)
    assert codes.shape == (rows, cols) and s.shape == (rows, scale_bytes(cols))
    assert (s[:, nb:] == 127).all(), "pad bytes"
    amax, e = block_amax(y), block_amax(err)
    got = s[:, :nb].astype(np.int64)
    # the scale of some magnitude within the error
    lo, hi = scale_of(np.maximum(amax - e, 0)), scale_of(amax + e)
    zero = amax + e == 0
    ok = np.where(zero, got == 127, (got >= np.where(amax - e <= 0, 1, lo)) & (got <= hi))
    assert ok.all(), f"scales off at {np.argwhere(~ok)[:4].tolist()}"
    sv = expand(s, cols)
    off = np.abs(CODE_VALUES[codes] * sv - y)
    # 448 may be exceeded by err where the scale is the smaller of two
    allowed = np.maximum(np.abs(y) * 2.0 ** -4, sv * 2.0 ** -10) + 2 * err + np.abs(y) * 2.0 ** -23
    assert (off <= allowed).all(), f"codes off by {(off / allowed).max()} of what is allowed"
