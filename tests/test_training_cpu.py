"""What the calls for the experts' gradients, low-rank adapters and gradient clipping refuse, found on the host
before anything is enqueued, the sizes they report and the table of gradients (CPU only: no call here reaches
the GPU)."""
import ctypes
import os

import pytest
import torch

import load_balancing_amd as mx
from test_binding_cpu import OnGpu, calls, one_gpu  # noqa: F401

vp, B, i64 = ctypes.c_void_p, ctypes.byref, ctypes.c_int64
FAKE = 0x10000000  # never dereferenced: every call below fails validation first, or has nothing to do
OK, SHAPE, NULL, MISALIGNED, WORKSPACE, ALIAS, ARG = 0, -1, -2, -3, -4, -6, -7


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mx.LIB_PATH):
        from load_balancing_amd import build
        build.build()
    return mx.lib()


def at(n):
    """A fake array of its own, far from the others."""
    return vp(FAKE * (n + 1))


def test_dx_refusals(L):
    s, n = mx.Shape(4, 16, 8, 2, 64), 256 * 128
    call = lambda plan=at(0), ws=at(1), Bs=2, inp=256, out=128, dy=at(2), wh=at(3), pool=at(4), st=2 * n, wo=n, \
        dx=at(5), sh=s: L.moonep_expert_gemm_dx(B(sh), plan, ws, Bs, inp, out, dy, wh, pool, i64(st), i64(wo), dx, None)  # noqa: E731
    assert call(sh=mx.Shape(3, 16, 8, 2, 64)) == SHAPE
    assert call(Bs=-1) == ARG and call(Bs=1 << 30) == ARG
    assert call(inp=0) == ARG and call(inp=32) == ARG and call(inp=-64) == ARG and call(out=64) == ARG and call(out=0) == ARG
    assert call(inp=(1 << 22) + 64, st=1 << 36, wo=0) == ARG and call(out=(1 << 22) + 128, st=1 << 36, wo=0) == ARG
    assert call(st=2 * n - 8) == ARG and call(wo=n + 8) == ARG and call(wo=-8) == ARG and call(wo=4) == ARG
    assert call(st=2 * n + 4) == ARG and call(st=-(1 << 63)) == ARG and call(st=1 << 40) == ARG and call(wo=(1 << 63) - 8) == ARG
    for k in ("plan", "ws", "dy", "wh", "pool", "dx"):
        assert call(**{k: None}) == NULL, k
    assert call(dy=vp(FAKE * 3 + 8)) == MISALIGNED and call(dx=vp(FAKE * 6 + 2)) == MISALIGNED
    assert call(wh=vp(FAKE * 4 + 8)) == MISALIGNED and call(plan=vp(FAKE + 2)) == MISALIGNED
    assert call(dx=at(2)) == ALIAS and call(dx=vp(FAKE * 4 + 64)) == ALIAS and call(dx=at(4)) == ALIAS
    assert call(dx=at(0)) == ALIAS and call(dx=at(1)) == ALIAS
    assert call(sh=mx.Shape(4, 16, 0, 2, 64), dy=None, dx=None) == OK  # no rows: nothing to do


def test_dw_refusals(L):
    s, n = mx.Shape(4, 16, 8, 2, 64), 256 * 128
    call = lambda plan=at(0), inp=256, out=128, x=at(1), dy=at(2), acc=0, G=n + 4, go=4, home=at(3), rep=at(4), \
        sh=s: L.moonep_expert_gemm_dw(B(sh), plan, inp, out, x, dy, acc, i64(G), i64(go), home, rep, None)  # noqa: E731
    assert call(sh=mx.Shape(3, 16, 8, 2, 64)) == SHAPE
    assert call(inp=96) == ARG and call(out=192) == ARG and call(inp=0) == ARG
    assert call(G=n) == ARG and call(go=5) == ARG and call(go=-1) == ARG and call(G=-1) == ARG
    assert call(G=-(1 << 63)) == ARG and call(G=(1 << 63) - 1) == ARG and call(go=(1 << 63) - 1) == ARG
    for k in ("plan", "x", "dy", "home", "rep"):
        assert call(**{k: None}) == NULL, k
    assert call(x=vp(FAKE * 2 + 8)) == MISALIGNED and call(dy=vp(FAKE * 3 + 4)) == MISALIGNED
    assert call(home=vp(FAKE * 4 + 2)) == MISALIGNED and call(rep=vp(FAKE * 5 + 1)) == MISALIGNED
    assert call(home=at(1)) == ALIAS and call(rep=at(2)) == ALIAS and call(rep=vp(FAKE * 4 + 64)) == ALIAS
    assert call(home=at(0)) == ALIAS
    assert call(sh=mx.Shape(4, 16, 0, 2, 64), x=None, dy=None, acc=1) == OK  # nothing to add


def adapters(**k):
    ad = dict(n=3, rank=16, in_dim=64, out_dim=72, stride=16 * 136, a_offset=0, b_offset=16 * 64)
    ad.update(k)
    return mx.Adapters(**ad)


def test_adapter_rules(L):
    s = mx.Shape(1, 4, 100, 1, 8)
    assert mx.moonep_adapter_workspace_bytes(s, adapters()) >= 100 * 16 * 4
    assert mx.moonep_adapter_bwd_workspace_bytes(s, adapters()) >= 100 * 16 * 4 + 3 * 16 * 136 * 4
    d = mx.Adapters(3, 16, 64, 72)  # by default a row holds the two matrices
    assert (d.stride, d.a_offset, d.b_offset) == (16 * 136, 0, 16 * 64)
    assert mx.moonep_adapter_workspace_bytes(s, adapters(a_offset=72 * 16, b_offset=0)) > 0  # in either order
    bad = [dict(n=0), dict(n=5), dict(n=-1), dict(rank=0), dict(rank=12), dict(rank=136), dict(rank=-8), dict(in_dim=60),
           dict(in_dim=0), dict(out_dim=4), dict(out_dim=-8), dict(in_dim=(1 << 22) + 8, stride=1 << 40, b_offset=1 << 39),
           dict(stride=16 * 136 - 8), dict(stride=16 * 136 + 4), dict(stride=-(1 << 63)), dict(stride=(1 << 63) - 8),
           dict(a_offset=-8), dict(a_offset=4), dict(b_offset=16 * 64 - 8), dict(b_offset=16 * 64 + 8),
           dict(a_offset=8, stride=16 * 140), dict(b_offset=(1 << 63) - 8), dict(a_offset=(1 << 63) - 8)]
    for k in bad:
        assert mx.moonep_adapter_workspace_bytes(s, adapters(**k)) == 0, k
        assert mx.moonep_adapter_bwd_workspace_bytes(s, adapters(**k)) == 0, k
        assert L.moonep_adapter(B(s), B(adapters(**k)), *[at(i) for i in range(9)], 1 << 30, None) == ARG, k
    for sh in (mx.Shape(2, 4, 100, 1, 8), mx.Shape(1, 4, 100, 2, 8), mx.Shape(1, 4, (1 << 30) + 1, 1, 8)):
        assert mx.moonep_adapter_workspace_bytes(sh, adapters()) == 0
        assert L.moonep_adapter(B(sh), B(adapters()), *[at(i) for i in range(9)], 1 << 30, None) == ARG
    assert mx.moonep_adapter_workspace_bytes(mx.Shape(3, 4, 100, 1, 8), adapters()) == 0
    assert L.moonep_adapter_workspace_bytes(B(s), None) == 0


def test_adapter_refusals(L):
    s, ad = mx.Shape(1, 4, 100, 1, 8), adapters()
    need = mx.moonep_adapter_workspace_bytes(s, ad)
    call = lambda ids=at(0), order=at(1), x=at(2), bank=at(3), scale=at(4), base=at(5), u=at(6), y=at(7), ws=at(8), \
        n=need, sh=s, a=ad: L.moonep_adapter(B(sh), B(a), ids, order, x, bank, scale, base, u, y, ws, n, None)  # noqa: E731
    assert L.moonep_adapter(B(s), None, *[at(i) for i in range(9)], need, None) == NULL
    for k in ("ids", "x", "bank", "scale", "base", "u", "y", "ws"):
        assert call(**{k: None}) == NULL, k
    for i, k in enumerate(("ids", "order", "x", "bank", "scale", "base", "u", "y", "ws")):
        off = 2 if k in ("ids", "order", "scale") else 8
        assert call(**{k: vp(FAKE * (i + 1) + off)}) == MISALIGNED, k
    assert call(n=need - 1) == WORKSPACE
    assert call(y=vp(FAKE * 6 + 16)) == ALIAS            # over base, but not base itself
    for k in range(5):
        assert call(y=at(k)) == ALIAS and call(u=at(k)) == ALIAS and call(ws=at(k)) == ALIAS, k
    assert call(u=at(5)) == ALIAS and call(u=at(7)) == ALIAS and call(ws=at(6)) == ALIAS and call(ws=vp(FAKE * 8 + 32)) == ALIAS
    assert call(base=at(7), u=at(7)) == ALIAS
    empty = mx.Shape(1, 4, 0, 1, 8)
    assert call(sh=empty, ids=None, order=None, x=None, base=None, u=None, y=None) == OK


def test_adapter_bwd_refusals(L):
    s, ad = mx.Shape(1, 4, 100, 1, 8), adapters()
    need = mx.moonep_adapter_bwd_workspace_bytes(s, ad)
    call = lambda ids=at(0), order=at(1), plan=at(2), x=at(3), u=at(4), dy=at(5), bank=at(6), scale=at(7), base=at(8), \
        dx=at(9), acc=0, db=at(10), ws=at(11), n=need, sh=s, a=ad: L.moonep_adapter_bwd(
            B(sh), B(a), ids, order, plan, x, u, dy, bank, scale, base, dx, acc, db, ws, n, None)  # noqa: E731
    for k in ("ids", "order", "plan", "x", "u", "dy", "bank", "scale", "ws"):
        assert call(**{k: None}) == NULL, k
    assert call(base=None) == NULL and call(dx=None) == NULL       # both or neither
    assert call(base=None, dx=None, db=None) == NULL               # nothing asked for
    for i, k in enumerate(("ids", "order", "plan", "x", "u", "dy", "bank", "scale", "base", "dx")):
        off = 2 if k in ("ids", "order", "plan", "scale") else 8
        assert call(**{k: vp(FAKE * (i + 1) + off)}) == MISALIGNED, k
    assert call(db=vp(FAKE * 11 + 4)) == MISALIGNED and call(ws=vp(FAKE * 12 + 8)) == MISALIGNED
    assert call(n=need - 1) == WORKSPACE
    assert call(dx=vp(FAKE * 9 + 16)) == ALIAS
    for k in range(8):
        assert call(dx=at(k)) == ALIAS and call(db=at(k)) == ALIAS and call(ws=at(k)) == ALIAS, k
    assert call(db=at(9)) == ALIAS and call(db=at(8)) == ALIAS and call(ws=at(10)) == ALIAS
    assert call(sh=mx.Shape(1, 4, 0, 1, 8), ids=None, order=None, x=None, u=None, dy=None, acc=1) == OK


def table(src, dst, counts, types, entries=None):
    n = len(counts)
    need = mx.moonep_grad_entries(counts)
    entries = need if entries is None else entries
    words = (ctypes.c_int64 * (4 * max(1, need, entries)))(*[-1] * (4 * max(1, need, entries)))
    U, I, T = ctypes.c_uint64 * n, ctypes.c_int64 * n, ctypes.c_int32 * n
    rc = mx.lib().moonep_grad_table(n, U(*src), U(*dst) if dst else None, I(*counts), T(*types), entries, words)
    return rc, [tuple(words[4 * i:4 * i + 4]) for i in range(max(need, entries, 0))]


def test_grad_table(L):
    run = mx.GRAD_RUN
    assert mx.moonep_grad_entries([]) == 0 and mx.moonep_grad_entries([0, 1, run, run + 1, 3 * run]) == 1 + 1 + 2 + 3
    assert mx.moonep_grad_entries([5, -1]) == -1 and mx.moonep_grad_entries([1 << 60]) == -1
    assert L.moonep_grad_entries(i64(-1), None) == -1 and L.moonep_grad_entries(i64(2), None) == -1
    rc, rows = table([1 << 20, 1 << 24, 0], None, [run + 3, 5, 0], [mx.F32, mx.BF16, mx.F32])
    assert rc == OK
    assert rows == [(1 << 20, 1 << 20, run, mx.F32), ((1 << 20) + 4 * run, (1 << 20) + 4 * run, 3, mx.F32),
                    (1 << 24, 1 << 24, 5, mx.BF16)]
    rc, rows = table([1 << 20, 1 << 24], [1 << 28, 1 << 24], [2, 5], [mx.F32, mx.BF16])
    assert rc == OK and rows == [(1 << 20, 1 << 28, 2, mx.F32), (1 << 24, 1 << 24, 5, mx.BF16)]
    # entries past the last run have no elements
    for counts, used in (([5], 1), ([], 0)):
        rc, rows = table([4096] * used, None, counts, [mx.F32] * used, entries=3)
        assert rc == OK and rows[used:] == [(0, 0, 0, 0)] * (3 - used)
    # neighbours that touch are apart
    assert table([4096, 4096 + 40], None, [10, 10], [mx.F32, mx.F32])[0] == OK


def test_grad_table_refusals(L):
    f, b = mx.F32, mx.BF16
    assert table([4096], None, [8], [2])[0] == ARG and table([4096], None, [8], [-1])[0] == ARG
    assert table([4098], None, [8], [f])[0] == MISALIGNED and table([4097], None, [8], [b])[0] == MISALIGNED
    assert table([4098], None, [8], [b])[0] == OK
    assert table([4096], [8194], [8], [f])[0] == MISALIGNED
    assert table([0], None, [8], [f])[0] == NULL and table([4096], [0], [8], [f])[0] == NULL
    assert table([4096], None, [8], [f], entries=0)[0] == WORKSPACE
    assert table([4096, 4096], None, [8, 8], [f, f])[0] == ALIAS            # the same tensor twice
    assert table([4096, 4096 + 28], None, [8, 8], [f, f])[0] == ALIAS
    assert table([4096 + 28, 4096], None, [8, 8], [f, f])[0] == ALIAS
    assert table([4096, 8192], [16384, 4096], [8, 8], [f, f])[0] == ALIAS   # an output on another's gradient
    assert table([4096, 8192], [16384, 16400], [8, 8], [f, f])[0] == ALIAS  # two outputs
    assert table([4096], [4100], [8], [f])[0] == ALIAS                      # over itself, but not itself
    assert L.moonep_grad_table(i64(-1), None, None, None, None, i64(0), None) == ARG
    assert L.moonep_grad_table(i64(1), None, None, None, None, i64(0), None) == NULL
    assert L.moonep_grad_table(i64(0), None, None, None, None, i64(0), None) == OK


def test_grad_call_refusals(L):
    norm = lambda n=4, t=at(0), ss=at(1), nm=at(2), ws=at(3), b=mx.GRAD_WORKSPACE_BYTES: \
        L.moonep_grad_norm(i64(n), t, ss, nm, ws, b, None)  # noqa: E731
    assert norm(n=-1) == ARG and norm(t=None) == NULL and norm(nm=None) == NULL and norm(ws=None) == NULL
    assert norm(t=vp(FAKE + 4)) == MISALIGNED and norm(ss=vp(FAKE * 2 + 4)) == MISALIGNED
    assert norm(nm=vp(FAKE * 3 + 2)) == MISALIGNED and norm(ws=vp(FAKE * 4 + 4)) == MISALIGNED
    assert norm(b=mx.GRAD_WORKSPACE_BYTES - 1) == WORKSPACE
    assert norm(nm=at(0)) == ALIAS and norm(ss=at(0)) == ALIAS and norm(ws=at(0)) == ALIAS and norm(nm=vp(FAKE * 4 + 8)) == ALIAS
    clip = lambda n=4, t=at(0), m=1.0, ss=at(1), nm=at(2), ws=at(3), b=mx.GRAD_WORKSPACE_BYTES: \
        L.moonep_grad_clip(i64(n), t, m, ss, nm, ws, b, None)  # noqa: E731
    for m in (-1.0, float("nan"), float("inf"), -float("inf")):
        assert clip(m=m) == ARG
    assert clip(n=-1) == ARG and clip(t=None) == NULL and clip(nm=None) == NULL
    assert clip(ss=None, ws=None) == NULL                          # one of the two
    assert clip(ss=None, b=mx.GRAD_WORKSPACE_BYTES - 1) == WORKSPACE
    assert clip(ws=vp(FAKE * 4 + 4)) == MISALIGNED and clip(ss=vp(FAKE * 2 + 4)) == MISALIGNED
    assert clip(nm=at(0)) == ALIAS and clip(nm=at(1)) == ALIAS and clip(ws=at(0)) == ALIAS and clip(ws=at(1)) == ALIAS
    assert mx.GRAD_WORKSPACE_BYTES == 16384 and mx.GRAD_RUN == 16384


def test_binding_checks(one_gpu, calls):  # noqa: F811
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    s, E, R, n = mx.Shape(2, 4, 8, 1, 8), 4, 2, 64 * 128
    words = 16 + 5 * 6 + 6 * 4 + 3 * 2
    arr = lambda *a: OnGpu(*a)  # noqa: E731
    mx._plan_words.cache_clear()
    orig, mx.moonep_plan_bytes = mx.moonep_plan_bytes, lambda shape: 4 * (16 + 5 * (shape.E + shape.R) + 6 * shape.E + 3 * shape.R)
    try:
        plan, ws = arr(words, i32), arr(E + R, i32)
        good = dict(d_y=arr(16 * 128, bf), w_home=arr(E * n, bf), pool=arr(2 * n, bf), d_x=arr(16 * 64, bf))
        dx = lambda **k: mx.moonep_expert_gemm_dx(  # noqa: E731
            s, plan, ws, 1, 64, 128, *[{**good, **k}[i] for i in ("d_y", "w_home", "pool")], n, 0, {**good, **k}["d_x"])
        dx()
        for k in good:
            for wrong in (arr(good[k].numel() + 8, bf), arr(good[k].numel(), f32), arr(good[k].numel(), bf, 1)):
                with pytest.raises(ValueError, match=k):
                    dx(**{k: wrong})
        dw = lambda home=arr(E * n, f32), rep=arr((E + R) * n, f32): mx.moonep_expert_gemm_dw(  # noqa: E731
            s, plan, 64, 128, arr(16 * 64, bf), arr(16 * 128, bf), True, n, 0, home, rep)
        dw()
        assert calls[-1][0] == "moonep_expert_gemm_dw" and calls[-1][1][6] == 1
        with pytest.raises(ValueError, match="home_grads"):
            dw(home=arr(E * n, bf))
        with pytest.raises(ValueError, match="replica_grads"):
            dw(rep=arr(E * n, f32))
        sa, ad = mx.Shape(1, 4, 10, 1, 8), mx.Adapters(3, 8, 16, 24)
        fwd = dict(ids=arr(10, i32), order=None, x=arr(160, bf), bank=arr(3 * 320, bf), scale=arr(3, f32),
                   base=arr(240, bf), u=arr(80, f32), y=arr(240, bf), workspace=arr(64, torch.uint8))
        mx.moonep_adapter(sa, ad, *fwd.values())
        assert calls[-1][1][3] is None
        for k in ("ids", "x", "bank", "scale", "base", "u", "y"):
            with pytest.raises(ValueError, match=k):
                mx.moonep_adapter(sa, ad, *{**fwd, k: arr(fwd[k].numel() + 1, fwd[k].dtype)}.values())
        with pytest.raises(ValueError, match="u"):
            mx.moonep_adapter(sa, ad, *{**fwd, "u": arr(80, bf)}.values())
        with pytest.raises(mx.MoonepError):
            mx.moonep_adapter(sa, ad, *{**fwd, "x": None}.values())
        bwd = dict(ids=arr(10, i32), order=arr(10, i32), plan=arr(16 + 25 + 24 + 3, i32), x=arr(160, bf),
                   u=arr(80, f32), d_y=arr(240, bf), bank=arr(3 * 320, bf), scale=arr(3, f32),
                   dx_base=arr(160, bf), d_x=arr(160, bf), accumulate=False, d_bank=arr(3 * 320, f32),
                   workspace=arr(64, torch.uint8))
        mx.moonep_adapter_bwd(sa, ad, *bwd.values())
        mx.moonep_adapter_bwd(sa, ad, *{**bwd, "order": None, "plan": None, "x": None, "u": None, "d_bank": None}.values())
        for k in ("order", "plan", "x", "u", "d_y", "d_x", "d_bank"):
            with pytest.raises(ValueError, match=k):
                mx.moonep_adapter_bwd(sa, ad, *{**bwd, k: arr(bwd[k].numel() + 1, bwd[k].dtype)}.values())
    finally:
        mx.moonep_plan_bytes = orig
        mx._plan_words.cache_clear()


def test_grad_table_binding_checks(one_gpu):  # noqa: F811
    """The table's tensors: type, size, device and number, before an address is used."""
    for grads, out in (([OnGpu(8, torch.float16)], None), ([OnGpu(8, torch.float32, 1)], None),
                       ([OnGpu(8, torch.float32)], [OnGpu(8, torch.bfloat16)]),
                       ([OnGpu(8, torch.float32)], [OnGpu(9, torch.float32)]), ([OnGpu(8, torch.float32)], [])):
        with pytest.raises(ValueError):
            mx.moonep_grad_table(grads, out)
