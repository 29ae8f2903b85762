"""Python binding of libmoonep, the gfx950 balanced expert-parallel hot path.

Thin ctypes marshalling over the C-ABI in include/moonep.h: every function
here has the name of the C entry point it calls, checks that the tensors it
is given match the shape (device, dtype, size, contiguity) and passes their
device pointers and the stream on.  All work runs in the HIP kernels of
libmoonep.so; there is no other implementation.  PyTorch supplies device
memory and streams only.

If libmoonep.so is not built, importing works but the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoonep.so")

MOONEP_OK = 0
ERRORS = {
    -1: "MOONEP_ERR_INVALID_SHAPE", -2: "MOONEP_ERR_NULL_PTR", -3: "MOONEP_ERR_MISALIGNED",
    -4: "MOONEP_ERR_WORKSPACE", -5: "MOONEP_ERR_HIP", -6: "MOONEP_ERR_ALIAS", -7: "MOONEP_ERR_ARG",
}
DEV_OK, DEV_BAD_EXPERT_ID = 0, 1
PLAN_HEADER = {"n_rep": 0, "n_spill": 1, "n_deficit": 2, "max_rep_rank": 3, "tmax": 4,
               "C": 5, "L": 6, "cap": 7}

EXPORTS = ("moonep_check_shape", "moonep_workspace_bytes", "moonep_plan_layout_of",
           "moonep_plan_bytes", "moonep_route_stats", "moonep_plan", "moonep_dispatch",
           "moonep_combine", "moonep_combine_bwd", "moonep_dispatch_bwd",
           "moonep_replica_grad_reduce", "moonep_weight_slots", "moonep_prefetch_weights",
           "moonep_expert_gemm", "moonep_read_error", "moonep_plan_largest_first",
           "moonep_plan_noalloc", "moonep_router_workspace_bytes", "moonep_router",
           "moonep_router_bwd", "moonep_scale_bytes", "moonep_rmsnorm_quant",
           "moonep_dispatch_quant", "moonep_quant_weights", "moonep_expert_gemm_quant",
           "moonep_expert_glu_quant")


class MoonepError(RuntimeError):
    def __init__(self, what: str, code: int):
        super().__init__(f"{what}: {ERRORS.get(code, code)}")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("S", ctypes.c_int32),
                ("K", ctypes.c_int32), ("H", ctypes.c_int32)]

    @property
    def N(self):
        return self.R * self.S

    @property
    def NK(self):
        return self.R * self.S * self.K

    @property
    def C(self):
        return self.S * self.K

    def __repr__(self):
        return f"Shape(R={self.R}, E={self.E}, S={self.S}, K={self.K}, H={self.H})"


SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
F32, BF16 = 0, 1


class RouterOpts(ctypes.Structure):
    """moonep_router_opts: score (SCORE_*), normalize, groups, logits_type (F32
    or BF16) and scale."""
    _fields_ = [("score", ctypes.c_int32), ("normalize", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("logits_type", ctypes.c_int32),
                ("scale", ctypes.c_float)]

    def __init__(self, score=SCORE_SOFTMAX, normalize=False, groups=1, logits_type=F32, scale=1.0):
        super().__init__(int(score), int(normalize), int(groups), int(logits_type), float(scale))


class PlanLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "words", "cap", "header", "rep_expert", "rep_host", "rep_count", "rep_spill_off",
        "rep_row_off", "spill", "keep", "home_row_off", "rep_first", "rep_cnt", "exp_rep_list",
        "load", "rank_rep_first", "rank_rep_cnt")]


_lib = None


def lib():
    """The loaded libmoonep.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m load_balancing_amd.build` (there is no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, VP, SZ, I64 = ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        I32, RO = ctypes.c_int32, ctypes.POINTER(RouterOpts)
        sig = {
            "moonep_check_shape": (ctypes.c_int, [P]),
            "moonep_workspace_bytes": (SZ, [P]),
            "moonep_plan_layout_of": (ctypes.c_int, [P, ctypes.POINTER(PlanLayout)]),
            "moonep_plan_bytes": (SZ, [P]),
            "moonep_route_stats": (ctypes.c_int, [P, VP, VP, VP, VP, SZ, VP]),
            "moonep_plan": (ctypes.c_int, [P, VP, VP, VP, SZ, VP, VP, VP, VP]),
            "moonep_plan_largest_first": (ctypes.c_int, [P, VP, VP, VP, SZ, VP, VP, VP, VP]),
            "moonep_dispatch": (ctypes.c_int, [P, VP, VP, VP, VP]),
            "moonep_combine": (ctypes.c_int, [P, VP, VP, VP, VP, VP]),
            "moonep_combine_bwd": (ctypes.c_int, [P, VP, VP, VP, VP, VP, VP, VP]),
            "moonep_dispatch_bwd": (ctypes.c_int, [P, VP, VP, VP, VP]),
            "moonep_replica_grad_reduce": (ctypes.c_int, [P, VP, I64, VP, VP, VP]),
            "moonep_weight_slots": (ctypes.c_int, [P, VP, ctypes.c_int32, VP, VP]),
            "moonep_prefetch_weights": (ctypes.c_int, [P, VP, VP, ctypes.c_int32, I64, VP, VP, VP]),
            "moonep_expert_gemm": (ctypes.c_int, [P, VP, VP, ctypes.c_int32, ctypes.c_int32,
                                                  ctypes.c_int32, VP, VP, VP, I64, I64, VP, VP]),
            "moonep_read_error": (ctypes.c_int, [VP, SZ, ctypes.POINTER(ctypes.c_int32), VP]),
            "moonep_plan_noalloc": (ctypes.c_int, [P, VP, VP, VP, VP, VP, VP, VP]),
            "moonep_router_workspace_bytes": (SZ, [P, RO]),
            "moonep_router": (ctypes.c_int, [P, RO, VP, VP, VP, VP, VP, VP, VP, SZ, VP]),
            "moonep_router_bwd": (ctypes.c_int, [P, RO, VP, VP, VP, VP, VP, VP, VP]),
            "moonep_scale_bytes": (SZ, [I32]),
            "moonep_rmsnorm_quant": (ctypes.c_int, [P, VP, VP, VP, ctypes.c_float, VP, VP, VP, VP,
                                                    VP]),
            "moonep_dispatch_quant": (ctypes.c_int, [P, VP, VP, VP, VP, VP, VP]),
            "moonep_quant_weights": (ctypes.c_int, [P, I32, I32, VP, I64, I64, VP, I64, I64, I64,
                                                    VP]),
            "moonep_expert_gemm_quant": (ctypes.c_int, [P, VP, VP, I32, I32, I32, VP, VP, VP, VP,
                                                        I64, I64, I64, VP, VP]),
            "moonep_expert_glu_quant": (ctypes.c_int, [P, VP, VP, I32, I32, I32, VP, VP, VP, VP,
                                                       I64, I64, I64, I64, I64, VP, VP, VP]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != MOONEP_OK:
        raise MoonepError(what, rc)


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_BF16_OK = ("bfloat16", "int16", "uint16")
_dtype_names = {}  # torch.dtype -> its name


def _dtype_name(dtype):
    name = _dtype_names.get(dtype)
    if name is None:
        name = _dtype_names[dtype] = str(dtype).replace("torch.", "")
    return name


def _dev(t, what, numel, kinds):
    """Device pointer of tensor t after checking device, dtype, size, layout."""
    if t is None:
        if numel == 0:
            return None
        raise MoonepError(what, -2)
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{what}: tensor must be on a GPU")
    if _dtype_name(t.dtype) not in kinds:
        raise ValueError(f"{what}: dtype {t.dtype} not in {kinds}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{what}: has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        torch = _torch()
        # The current stream's handle without a Stream object built for it, where torch
        # has its internal accessor; that one is no public name.
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        return raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t):
    return t.numel() * t.element_size()


def _current_device():
    return _torch().cuda.current_device()


def _arg(dev, t, what, numel, kinds):
    """_dev for a tensor that has to be on device dev, the current one, whose
    stream the call takes; kinds None: numel bytes of any dtype."""
    if t is None or type(t) is int:
        return _dev(t, what, numel, kinds)
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, must be on a GPU, the current device")
    if kinds is None:
        return _dev_bytes(t, what, numel)
    if _dtype_names.get(t.dtype) not in kinds or not t.is_contiguous() or t.numel() != numel:
        return _dev(t, what, numel, kinds)  # says what is wrong (or has not seen the dtype yet)
    return t.data_ptr()


@functools.lru_cache(maxsize=None)
def _plan_words(E, R):
    return moonep_plan_bytes(Shape(R, E, 0, 1, 8)) // 4


def _scale_row(cols):
    return 4 * -(-cols // 512)


# ---------------------------------------------------------------------------
# the C-ABI, one Python function per entry point
# ---------------------------------------------------------------------------

def moonep_check_shape(shape: Shape) -> int:
    return lib().moonep_check_shape(ctypes.byref(shape))


def moonep_workspace_bytes(shape: Shape) -> int:
    return lib().moonep_workspace_bytes(ctypes.byref(shape))


def moonep_plan_bytes(shape: Shape) -> int:
    return lib().moonep_plan_bytes(ctypes.byref(shape))


def moonep_plan_layout_of(shape: Shape) -> PlanLayout:
    lay = PlanLayout()
    _check(lib().moonep_plan_layout_of(ctypes.byref(shape), ctypes.byref(lay)),
           "moonep_plan_layout_of")
    return lay


def moonep_route_stats(shape, topk_idx, expert_counts, maxvio, workspace, stream=None):
    _check(lib().moonep_route_stats(
        ctypes.byref(shape), _dev(topk_idx, "topk_idx", shape.NK, ("int32",)),
        _dev(expert_counts, "expert_counts", shape.E, ("int32",)),
        _dev(maxvio, "maxvio", 1, ("float32",)),
        _dev(workspace, "workspace", workspace.numel(), ("uint8",)), _nbytes(workspace),
        _stream(stream)), "moonep_route_stats")


def moonep_plan(shape, topk_idx, expert_counts, workspace, plan, slot_of, src_of_slot, stream=None):
    _check(lib().moonep_plan(
        ctypes.byref(shape), _dev(topk_idx, "topk_idx", shape.NK, ("int32",)),
        _dev(expert_counts, "expert_counts", shape.E, ("int32",)),
        _dev(workspace, "workspace", workspace.numel(), ("uint8",)), _nbytes(workspace),
        _dev(plan, "plan", moonep_plan_bytes(shape) // 4, ("int32",)),
        _dev(slot_of, "slot_of", shape.NK, ("int32",)),
        _dev(src_of_slot, "src_of_slot", shape.NK, ("int32",)), _stream(stream)), "moonep_plan")


def moonep_plan_largest_first(shape, topk_idx, expert_counts, workspace, plan, slot_of,
                              src_of_slot, stream=None):
    _check(lib().moonep_plan_largest_first(
        ctypes.byref(shape), _dev(topk_idx, "topk_idx", shape.NK, ("int32",)),
        _dev(expert_counts, "expert_counts", shape.E, ("int32",)),
        _dev(workspace, "workspace", workspace.numel(), ("uint8",)), _nbytes(workspace),
        _dev(plan, "plan", moonep_plan_bytes(shape) // 4, ("int32",)),
        _dev(slot_of, "slot_of", shape.NK, ("int32",)),
        _dev(src_of_slot, "src_of_slot", shape.NK, ("int32",)), _stream(stream)),
        "moonep_plan_largest_first")


def moonep_plan_noalloc(shape, topk_idx, expert_counts, maxvio, plan, slot_of, src_of_slot,
                        stream=None):
    _check(lib().moonep_plan_noalloc(
        ctypes.byref(shape), _dev(topk_idx, "topk_idx", shape.NK, ("int32",)),
        _dev(expert_counts, "expert_counts", shape.E, ("int32",)),
        _dev(maxvio, "maxvio", 1, ("float32",)),
        _dev(plan, "plan", moonep_plan_bytes(shape) // 4, ("int32",)),
        _dev(slot_of, "slot_of", shape.NK, ("int32",)),
        _dev(src_of_slot, "src_of_slot", shape.NK, ("int32",)), _stream(stream)),
        "moonep_plan_noalloc")


def moonep_dispatch(shape, x, slot_of, buf, stream=None):
    _check(lib().moonep_dispatch(
        ctypes.byref(shape), _dev(x, "x", shape.N * shape.H, _BF16_OK),
        _dev(slot_of, "slot_of", shape.NK, ("int32",)),
        _dev(buf, "buf", shape.NK * shape.H, _BF16_OK), _stream(stream)), "moonep_dispatch")


def moonep_combine(shape, expert_out, gates, slot_of, y, stream=None):
    _check(lib().moonep_combine(
        ctypes.byref(shape), _dev(expert_out, "expert_out", shape.NK * shape.H, _BF16_OK),
        _dev(gates, "gates", shape.NK, ("float32",)),
        _dev(slot_of, "slot_of", shape.NK, ("int32",)),
        _dev(y, "y", shape.N * shape.H, _BF16_OK), _stream(stream)), "moonep_combine")


def moonep_combine_bwd(shape, dy, expert_out, gates, slot_of, d_out, d_gates, stream=None):
    _check(lib().moonep_combine_bwd(
        ctypes.byref(shape), _dev(dy, "dy", shape.N * shape.H, _BF16_OK),
        _dev(expert_out, "expert_out", shape.NK * shape.H, _BF16_OK),
        _dev(gates, "gates", shape.NK, ("float32",)),
        _dev(slot_of, "slot_of", shape.NK, ("int32",)),
        _dev(d_out, "d_out", shape.NK * shape.H, _BF16_OK),
        _dev(d_gates, "d_gates", shape.NK, ("float32",)), _stream(stream)), "moonep_combine_bwd")


def moonep_dispatch_bwd(shape, d_buf, slot_of, dx, stream=None):
    _check(lib().moonep_dispatch_bwd(
        ctypes.byref(shape), _dev(d_buf, "d_buf", shape.NK * shape.H, _BF16_OK),
        _dev(slot_of, "slot_of", shape.NK, ("int32",)),
        _dev(dx, "dx", shape.N * shape.H, _BF16_OK), _stream(stream)), "moonep_dispatch_bwd")


def moonep_replica_grad_reduce(shape, plan, G, home_grads, replica_grads, stream=None):
    _check(lib().moonep_replica_grad_reduce(
        ctypes.byref(shape), _dev(plan, "plan", moonep_plan_bytes(shape) // 4, ("int32",)),
        int(G), _dev(home_grads, "home_grads", shape.E * G, ("float32",)),
        _dev(replica_grads, "replica_grads", (shape.E + shape.R) * G, ("float32",)),
        _stream(stream)), "moonep_replica_grad_reduce")


def moonep_weight_slots(shape, plan, B, wslot, stream=None):
    _check(lib().moonep_weight_slots(
        ctypes.byref(shape), _dev(plan, "plan", moonep_plan_bytes(shape) // 4, ("int32",)),
        int(B), _dev(wslot, "wslot", shape.E + shape.R, ("int32",)), _stream(stream)),
        "moonep_weight_slots")


def _dev_bytes(t, what, nbytes):
    """Device pointer of a contiguous tensor of any dtype holding exactly nbytes."""
    if t is None:
        if nbytes == 0:
            return None
        raise MoonepError(what, -2)
    if not t.is_cuda:
        raise ValueError(f"{what}: tensor must be on a GPU")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if _nbytes(t) != nbytes:
        raise ValueError(f"{what}: has {_nbytes(t)} bytes, needs {nbytes}")
    return t.data_ptr()


def moonep_prefetch_weights(shape, plan, wslot, B, wbytes, w_home, pool, stream=None):
    """pool [R*B, wbytes] gets each slotted replica's row of w_home [E, wbytes]."""
    _check(lib().moonep_prefetch_weights(
        ctypes.byref(shape), _dev(plan, "plan", moonep_plan_bytes(shape) // 4, ("int32",)),
        _dev(wslot, "wslot", shape.E + shape.R, ("int32",)), int(B), int(wbytes),
        _dev_bytes(w_home, "w_home", shape.E * wbytes),
        _dev_bytes(pool, "pool", shape.R * B * wbytes), _stream(stream)),
        "moonep_prefetch_weights")


def moonep_expert_gemm(shape, plan, wslot, B, in_dim, out_dim, x, w_home, pool, w_stride,
                       w_offset, y, stream=None):
    """y [R*S*K, out_dim] = each buffer row of x [R*S*K, in_dim] times its
    segment's weights; w_home [E, w_stride] and pool [R*B, w_stride] bf16."""
    _check(lib().moonep_expert_gemm(
        ctypes.byref(shape), _dev(plan, "plan", moonep_plan_bytes(shape) // 4, ("int32",)),
        _dev(wslot, "wslot", shape.E + shape.R, ("int32",)), int(B), int(in_dim), int(out_dim),
        _dev(x, "x", shape.NK * in_dim, _BF16_OK),
        _dev_bytes(w_home, "w_home", shape.E * w_stride * 2),
        _dev_bytes(pool, "pool", shape.R * B * w_stride * 2), int(w_stride), int(w_offset),
        _dev(y, "y", shape.NK * out_dim, _BF16_OK), _stream(stream)), "moonep_expert_gemm")


def moonep_router_workspace_bytes(shape, opts: RouterOpts) -> int:
    return lib().moonep_router_workspace_bytes(ctypes.byref(shape), ctypes.byref(opts))


def _logit_kinds(opts):
    return _BF16_OK if opts.logits_type == BF16 else ("float32",)


def moonep_router(shape, opts, logits, topk_idx, gates, counts=None, prob_sum=None, loss=None,
                  workspace=None, stream=None):
    """topk_idx and gates [R*S*K] of logits [R*S, E]; with counts and prob_sum
    [groups, E], loss [1] and a workspace also the balance loss."""
    dev = _current_device()
    some = not (counts is None and prob_sum is None and loss is None and workspace is None)
    tab = opts.groups * shape.E if some else 0
    _check(lib().moonep_router(
        ctypes.byref(shape), ctypes.byref(opts),
        _arg(dev, logits, "logits", shape.N * shape.E, _logit_kinds(opts)),
        _arg(dev, topk_idx, "topk_idx", shape.NK, ("int32",)),
        _arg(dev, gates, "gates", shape.NK, ("float32",)),
        _arg(dev, counts, "counts", tab, ("int32",)),
        _arg(dev, prob_sum, "prob_sum", tab, ("float32",)),
        _arg(dev, loss, "loss", 1 if some else 0, ("float32",)),
        _arg(dev, workspace, "workspace", workspace.numel() if workspace is not None else int(some),
             ("uint8",)),
        _nbytes(workspace) if workspace is not None else 0, _stream(stream)), "moonep_router")


def moonep_router_bwd(shape, opts, logits, topk_idx, counts, d_gates, d_loss, d_logits,
                      stream=None):
    """d_logits [R*S, E] from d_gates [R*S*K] (None: 0) and d_loss [1] with the
    forward's counts (both None: no loss)."""
    dev = _current_device()
    n = shape.N * shape.E
    _check(lib().moonep_router_bwd(
        ctypes.byref(shape), ctypes.byref(opts), _arg(dev, logits, "logits", n, _logit_kinds(opts)),
        _arg(dev, topk_idx, "topk_idx", shape.NK, ("int32",)),
        _arg(dev, counts, "counts", 0 if counts is None else opts.groups * shape.E, ("int32",)),
        _arg(dev, d_gates, "d_gates", 0 if d_gates is None else shape.NK, ("float32",)),
        _arg(dev, d_loss, "d_loss", 0 if d_loss is None else 1, ("float32",)),
        _arg(dev, d_logits, "d_logits", n, _logit_kinds(opts)), _stream(stream)),
        "moonep_router_bwd")


_CODES = ("float8_e4m3fn", "uint8")
_SCALES = ("float8_e8m0fnu", "uint8")


def moonep_scale_bytes(cols: int) -> int:
    """Bytes of the scales of one 8-bit row of `cols` columns."""
    return lib().moonep_scale_bytes(int(cols))


def moonep_rmsnorm_quant(shape, x, res, weight, eps, res_out, y_out, y8, ys, stream=None):
    """res_out = x + res (both None: x alone), y8 and ys its RMS norm times weight
    [H] as 8-bit rows, y_out (or None) the same in bf16."""
    dev = _current_device()
    n = shape.N * shape.H
    _check(lib().moonep_rmsnorm_quant(
        ctypes.byref(shape), _arg(dev, x, "x", n, _BF16_OK),
        _arg(dev, res, "res", 0 if res is None else n, _BF16_OK),
        _arg(dev, weight, "weight", shape.H, _BF16_OK), float(eps),
        _arg(dev, res_out, "res_out", 0 if res_out is None else n, _BF16_OK),
        _arg(dev, y_out, "y_out", 0 if y_out is None else n, _BF16_OK),
        _arg(dev, y8, "y8", n, _CODES),
        _arg(dev, ys, "ys", shape.N * _scale_row(shape.H), _SCALES), _stream(stream)),
        "moonep_rmsnorm_quant")


def moonep_dispatch_quant(shape, x8, xs, slot_of, buf8, bufs, stream=None):
    """buf8 [R*S*K, H] and bufs get every token's codes and scales at its slots."""
    dev = _current_device()
    sb = _scale_row(shape.H)
    _check(lib().moonep_dispatch_quant(
        ctypes.byref(shape), _arg(dev, x8, "x8", shape.N * shape.H, _CODES),
        _arg(dev, xs, "xs", shape.N * sb, _SCALES),
        _arg(dev, slot_of, "slot_of", shape.NK, ("int32",)),
        _arg(dev, buf8, "buf8", shape.NK * shape.H, _CODES),
        _arg(dev, bufs, "bufs", shape.NK * sb, _SCALES),
        _stream(stream)), "moonep_dispatch_quant")


def moonep_quant_weights(shape, in_dim, out_dim, w, w_stride, w_offset, w8, w8_stride, code_offset,
                         scale_offset, stream=None):
    """The [out_dim, in_dim] bf16 matrices at element w_offset of w [E, w_stride]
    to codes and scales inside the weight rows of w8 [E, w8_stride] bytes."""
    dev = _current_device()
    _check(lib().moonep_quant_weights(
        ctypes.byref(shape), int(in_dim), int(out_dim),
        _arg(dev, w, "w", shape.E * w_stride, _BF16_OK), int(w_stride), int(w_offset),
        _arg(dev, w8, "w8", shape.E * w8_stride, None), int(w8_stride), int(code_offset),
        int(scale_offset), _stream(stream)), "moonep_quant_weights")


def moonep_expert_gemm_quant(shape, plan, wslot, B, in_dim, out_dim, x8, xs, w_home, pool, w_stride,
                             code_offset, scale_offset, y, stream=None):
    """y [R*S*K, out_dim] bf16 = each 8-bit buffer row times its segment's 8-bit
    weights; w_home [E, w_stride] and pool [R*B, w_stride] bytes."""
    dev = _current_device()
    _check(lib().moonep_expert_gemm_quant(
        ctypes.byref(shape), _arg(dev, plan, "plan", _plan_words(shape.E, shape.R), ("int32",)),
        _arg(dev, wslot, "wslot", shape.E + shape.R, ("int32",)), int(B), int(in_dim), int(out_dim),
        _arg(dev, x8, "x8", shape.NK * in_dim, _CODES),
        _arg(dev, xs, "xs", shape.NK * _scale_row(in_dim), _SCALES),
        _arg(dev, w_home, "w_home", shape.E * w_stride, None),
        _arg(dev, pool, "pool", shape.R * B * w_stride, None), int(w_stride), int(code_offset),
        int(scale_offset), _arg(dev, y, "y", shape.NK * out_dim, _BF16_OK), _stream(stream)),
        "moonep_expert_gemm_quant")


def moonep_expert_glu_quant(shape, plan, wslot, B, in_dim, mid_dim, x8, xs, w_home, pool, w_stride,
                            gate_code_offset, gate_scale_offset, up_code_offset, up_scale_offset,
                            h8, hs, stream=None):
    """h8 [R*S*K, mid_dim] and hs: silu of the gate projection times the up
    projection of each 8-bit buffer row, as 8-bit rows."""
    dev = _current_device()
    _check(lib().moonep_expert_glu_quant(
        ctypes.byref(shape), _arg(dev, plan, "plan", _plan_words(shape.E, shape.R), ("int32",)),
        _arg(dev, wslot, "wslot", shape.E + shape.R, ("int32",)), int(B), int(in_dim), int(mid_dim),
        _arg(dev, x8, "x8", shape.NK * in_dim, _CODES),
        _arg(dev, xs, "xs", shape.NK * _scale_row(in_dim), _SCALES),
        _arg(dev, w_home, "w_home", shape.E * w_stride, None),
        _arg(dev, pool, "pool", shape.R * B * w_stride, None), int(w_stride), int(gate_code_offset),
        int(gate_scale_offset), int(up_code_offset), int(up_scale_offset),
        _arg(dev, h8, "h8", shape.NK * mid_dim, _CODES),
        _arg(dev, hs, "hs", shape.NK * _scale_row(mid_dim), _SCALES), _stream(stream)),
        "moonep_expert_glu_quant")


def moonep_read_error(workspace, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(lib().moonep_read_error(_dev(workspace, "workspace", workspace.numel(), ("uint8",)),
                                   _nbytes(workspace), ctypes.byref(code), _stream(stream)),
           "moonep_read_error")
    return code.value


# ---------------------------------------------------------------------------
# static buffers of one MoE layer (allocated once; sizes depend on the shape only)
# ---------------------------------------------------------------------------

@dataclass
class Buffers:
    shape: Shape
    workspace: object      # uint8 [moonep_workspace_bytes], zeroed once
    expert_counts: object  # int32 [E]
    maxvio: object         # fp32 [1]
    plan: object           # int32 [moonep_plan_bytes / 4]
    slot_of: object        # int32 [R*S*K]
    src_of_slot: object    # int32 [R*S*K]
    buf: object            # bf16 [R*S*K, H]: the R per-rank [S*K, H] buffers

    def plan_fields(self) -> dict:
        """Plan table as named host int arrays (reads the device)."""
        lay = moonep_plan_layout_of(self.shape)
        p = self.plan.cpu().numpy()
        E, R, cap = self.shape.E, self.shape.R, lay.cap
        sizes = {"rep_expert": cap, "rep_host": cap, "rep_count": cap, "rep_spill_off": cap,
                 "rep_row_off": cap, "spill": E, "keep": E, "home_row_off": E, "rep_first": E,
                 "rep_cnt": E, "exp_rep_list": E, "load": R, "rank_rep_first": R,
                 "rank_rep_cnt": R}
        out = {k: p[getattr(lay, k):getattr(lay, k) + n] for k, n in sizes.items()}
        out.update({k: int(p[lay.header + i]) for k, i in PLAN_HEADER.items()})
        return out


def allocate(shape: Shape, device="cuda") -> Buffers:
    torch = _torch()
    _check(moonep_check_shape(shape), "allocate")
    ws = torch.zeros(moonep_workspace_bytes(shape), dtype=torch.uint8, device=device)
    return Buffers(
        shape=shape, workspace=ws,
        expert_counts=torch.empty(shape.E, dtype=torch.int32, device=device),
        maxvio=torch.empty(1, dtype=torch.float32, device=device),
        plan=torch.empty(moonep_plan_bytes(shape) // 4, dtype=torch.int32, device=device),
        slot_of=torch.empty(shape.NK, dtype=torch.int32, device=device),
        src_of_slot=torch.empty(shape.NK, dtype=torch.int32, device=device),
        buf=torch.empty((shape.NK, shape.H), dtype=torch.bfloat16, device=device),
    )


def plan_step(b: Buffers, topk_idx, stream=None, largest_first=False):
    """route_stats then plan (moonep_plan, or moonep_plan_largest_first):
    counts, maxvio, the plan and both slot maps."""
    moonep_route_stats(b.shape, topk_idx, b.expert_counts, b.maxvio, b.workspace, stream)
    planner = moonep_plan_largest_first if largest_first else moonep_plan
    planner(b.shape, topk_idx, b.expert_counts, b.workspace, b.plan, b.slot_of, b.src_of_slot,
            stream)
