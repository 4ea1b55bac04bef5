"""Python binding of the jetq C ABI (``include/jetq.h``).

Argument marshalling only: every function passes device pointers, sizes and
the current CUDA stream to ``_build/libjetq.so`` and raises ``JetqError`` on a
non-OK status.  PyTorch supplies device memory and streams.  There is no CPU
fallback: without the compiled library every call raises.

The ``jetq_*`` functions mirror the C entry points one to one.  The short
helpers below them (``quant_act``, ``quant_weight``, ``quant_mx``, ``fprop``,
``dgrad``, ``wgrad``) only allocate the output tensors with torch and call the
matching ``jetq_*`` function.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libjetq.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_MISALIGNED, ERR_ARCH, ERR_CUDA, ERR_TIMEOUT = range(7)
RECIPE_BLOCK128, RECIPE_MXFP8, RECIPE_BLOCK128_POW2 = 0, 1, 2
PATH_AUTO, PATH_TRAIN, PATH_DECODE = 0, 1, 2
GEMM_FPROP, GEMM_DGRAD, GEMM_WGRAD = 0, 1, 2
OUT_F32, OUT_BF16 = 0, 1
NORM_LAYER, NORM_RMS = 0, 1
POLICY_TOKEN, POLICY_SEGMENT = 0, 1
POLICY_MEAN_TOKENS, POLICY_MEAN_SEGMENTS, POLICY_SUM = 0, 1, 2

_lock = threading.Lock()
_lib = None


class JetqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"jetq CUDA library missing ({LIB_PATH}); build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        sig = {
            "jetq_status_string": (ctypes.c_char_p, [I32]),
            "jetq_version": (I32, []),
            "jetq_check_device_error": (I32, [P]),
            "jetq_selftest_bounded_wait": (I32, [ctypes.c_uint64, P, P]),
            "jetq_colcopy_capacity": (I64, [I64, I32]),
            "jetq_mx_scale_bytes": (I64, [I64, I64]),
            "jetq_quant_act_1x128": (I32, [P, I64, I64, I64, P, P, P, P, I64, P, I32, P]),
            "jetq_quant_act_1x128_rmsnorm": (I32, [P, I64, I64, I64, P, ctypes.c_float, P, P, P, P, P, I64, P, I32,
                                                   P]),
            "jetq_quant_act_1x128_swiglu": (I32, [P, P, I64, I64, I64, I64, P, P, P, P, I64, P, I32, P]),
            "jetq_quant_w_128x128": (I32, [P, I64, I64, I64, P, P, P, P, P]),
            "jetq_amax_bf16": (I32, [P, I64, I64, I64, P, P]),
            "jetq_quant_nvfp4": (I32, [P, I64, I64, I64, P, P, P, P, P]),
            "jetq_dequant_nvfp4_bf16": (I32, [P, P, P, I32, I64, I64, P, I64, P]),
            "jetq_quant_mx32": (I32, [P, I64, I64, I64, P, P, P, P, I64, P, I32, P]),
            "jetq_quant_act_1x128_pow2": (I32, [P, I64, I64, I64, P, P, P, P, I64, P, I32, P]),
            "jetq_quant_w_128x128_pow2": (I32, [P, I64, I64, I64, P, P, P, P, P]),
            "jetq_requant_col_from_row": (I32, [P, P, I64, I64, P, P, I64, P, I32, P]),
            "jetq_dequant_bf16": (I32, [P, P, I64, I64, I32, P, I64, P]),
            "jetq_gemm_fprop": (I32, [I32, P, P, P, P, I64, I64, I64, P, I32, I64, I32, P]),
            "jetq_decode_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64]),
            "jetq_gemm_fprop_ws": (I32, [I32, P, P, P, P, I64, I64, I64, P, I32, I64, P, ctypes.c_size_t, I32, P]),
            "jetq_gemm_fprop_noalloc": (I32, [P, P, P, P, I64, I64, I64, P, I32, I64, P]),
            "jetq_gemm_dgrad": (I32, [I32, P, P, P, P, I64, I64, I64, P, I32, I64, P]),
            "jetq_gemm_wgrad": (I32, [I32, P, P, P, P, I64, I64, I64, I64, P, I64, I32, P]),
            "jetq_gemm_grouped": (I32, [I32, I32, P, P, P, P, I64, I64, I64, I64, P, I32, P, I32, I64, I32, P]),
            "jetq_nvfp4_atom_bytes": (I64, [I64, I64]),
            "jetq_nvfp4_scale_atoms": (I32, [P, I64, I64, P, P]),
            "jetq_gemm_nvfp4": (I32, [P, P, P, I32, P, P, P, I64, I64, I64, P, I32, I64, P]),
            "jetq_gemv_nvfp4": (I32, [P, P, P, I64, I64, P, I64, I64, P, I32, I64, P]),
            "jetq_norm_fwd": (I32, [I32, I32, P, I64, I64, I64, P, P, F32, P, I64, P, P, P]),
            "jetq_norm_bwd_workspace_bytes": (ctypes.c_size_t, [I32, I64, I64]),
            "jetq_norm_bwd": (I32, [I32, I32, P, I64, P, I64, I64, I64, P, P, P, P, I64, P, P, P, ctypes.c_size_t,
                                    P]),
            "jetq_linear_ce_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64]),
            "jetq_linear_ce_fwd": (I32, [P, I64, I64, I64, P, I64, I64, P, F32, P, P, P, ctypes.c_size_t, P]),
            "jetq_linear_ce_bwd_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I32]),
            "jetq_linear_ce_bwd": (I32, [P, I64, I64, I64, P, I64, I64, P, F32, P, P, P, I64, P, I32, I64, I32, P,
                                         ctypes.c_size_t, P]),
            "jetq_linear_distill_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I64]),
            "jetq_linear_distill_fwd": (I32, [P, I64, I64, I64, P, I64, I64, P, I64, P, I64, I64, I32, F32, P, P, P, P,
                                              ctypes.c_size_t, P]),
            "jetq_linear_distill_bwd_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I64, I32]),
            "jetq_linear_distill_bwd": (I32, [P, I64, I64, I64, P, I64, I64, P, I64, P, I64, I64, I32, F32, P, P, P, P,
                                              I64, P, I32, I64, I32, P, ctypes.c_size_t, P]),
            "jetq_moe_nvfp4_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I64, I64]),
            "jetq_moe_nvfp4": (I32, [P, I64, I64, I64, P, I64, I64, I64, I32, P, P, P, I64, P, P, P, P, I32, I64, P, P,
                                     P, ctypes.c_size_t, P]),
            "jetq_policy_loss_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
            "jetq_policy_loss_fwd": (I32, [P, P, P, P, I32, P, I64, P, I64, I32, I32, F32, F32, F32, F32, F32, P, P, P,
                                           ctypes.c_size_t, P]),
            "jetq_policy_loss_bwd": (I32, [P, P, P, P, I32, P, I64, P, I64, I32, I32, F32, F32, F32, F32, F32, P, P, P,
                                           P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        return L


def status_string(status: int) -> str:
    try:
        return lib().jetq_status_string(int(status)).decode()
    except RuntimeError:
        return "unknown"


def _p(t):
    return None if t is None else t.data_ptr()


def _s(stream):
    # the raw handle of torch.cuda.current_stream(), without building the stream object on every call
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def _bytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def _check(status: int, where: str):
    if status != OK:
        raise JetqError(status, where)


# ------------------------------------------------------------------ C entry points

def jetq_version() -> int:
    return int(lib().jetq_version())


def jetq_check_device_error(stream=None) -> int:
    return int(lib().jetq_check_device_error(_s(stream)))


def jetq_selftest_bounded_wait(limit_ns: int, elapsed_ns, stream=None) -> int:
    """Launch the bounded-wait diagnostic; elapsed_ns: int64 CUDA tensor of 2."""
    return int(lib().jetq_selftest_bounded_wait(int(limit_ns), _p(elapsed_ns), _s(stream)))


def jetq_colcopy_capacity(n: int, nseg: int = 1) -> int:
    return int(lib().jetq_colcopy_capacity(n, nseg))


def jetq_mx_scale_bytes(rows: int, k: int) -> int:
    return int(lib().jetq_mx_scale_bytes(rows, k))


def jetq_quant_act_1x128(x, q_row, s_row, q_col, s_col, ldq_col, seg_offsets=None, nseg=0, stream=None):
    n, c = x.shape
    _check(lib().jetq_quant_act_1x128(_p(x), n, c, x.stride(0), _p(q_row), _p(s_row), _p(q_col), _p(s_col),
                                      ldq_col, _p(seg_offsets), nseg, _s(stream)), "jetq_quant_act_1x128")


def jetq_quant_act_1x128_rmsnorm(x, w, eps, rstd, q_row, s_row, q_col, s_col, ldq_col, seg_offsets=None, nseg=0,
                                 stream=None):
    n, c = x.shape
    _check(lib().jetq_quant_act_1x128_rmsnorm(_p(x), n, c, x.stride(0), _p(w), float(eps), _p(rstd), _p(q_row),
                                              _p(s_row), _p(q_col), _p(s_col), ldq_col, _p(seg_offsets), nseg,
                                              _s(stream)), "jetq_quant_act_1x128_rmsnorm")


def jetq_quant_act_1x128_swiglu(gate, up, q_row, s_row, q_col, s_col, ldq_col, seg_offsets=None, nseg=0, stream=None):
    n, c = gate.shape
    assert up.shape == gate.shape
    _check(lib().jetq_quant_act_1x128_swiglu(_p(gate), _p(up), n, c, gate.stride(0), up.stride(0), _p(q_row),
                                             _p(s_row), _p(q_col), _p(s_col), ldq_col, _p(seg_offsets), nseg,
                                             _s(stream)), "jetq_quant_act_1x128_swiglu")


def jetq_amax_bf16(x, amax, stream=None):
    r, c = x.shape
    _check(lib().jetq_amax_bf16(_p(x), r, c, x.stride(0), _p(amax), _s(stream)), "jetq_amax_bf16")


def jetq_quant_nvfp4(x, q, sb, sg, scope_amax=None, stream=None):
    r, c = x.shape
    _check(lib().jetq_quant_nvfp4(_p(x), r, c, x.stride(0), _p(scope_amax), _p(q), _p(sb), _p(sg), _s(stream)),
           "jetq_quant_nvfp4")


def jetq_dequant_nvfp4_bf16(q, sb, sg, per_row, out, stream=None):
    r, c = out.shape
    _check(lib().jetq_dequant_nvfp4_bf16(_p(q), _p(sb), _p(sg), int(per_row), r, c, _p(out), out.stride(0),
                                         _s(stream)), "jetq_dequant_nvfp4_bf16")


def jetq_nvfp4_atom_bytes(rows: int, k: int) -> int:
    return int(lib().jetq_nvfp4_atom_bytes(rows, k))


def jetq_nvfp4_scale_atoms(sb, rows, k, atoms, stream=None):
    _check(lib().jetq_nvfp4_scale_atoms(_p(sb), rows, k, _p(atoms), _s(stream)), "jetq_nvfp4_scale_atoms")


def jetq_gemm_nvfp4(qa, sfa, sga, per_row_a, qb, sfb, sgb, m, n, k, out, stream=None):
    _check(lib().jetq_gemm_nvfp4(_p(qa), _p(sfa), _p(sga), int(per_row_a), _p(qb), _p(sfb), _p(sgb), m, n, k,
                                 _p(out), _out_dtype(out), out.stride(0), _s(stream)), "jetq_gemm_nvfp4")


def jetq_quant_w_128x128(w, q, s, qT=None, sT=None, stream=None):
    d, c = w.shape
    _check(lib().jetq_quant_w_128x128(_p(w), d, c, w.stride(0), _p(q), _p(s), _p(qT), _p(sT), _s(stream)),
           "jetq_quant_w_128x128")


def jetq_quant_mx32(x, q_row, e8_row, q_col, e8_col, ldq_col, seg_offsets=None, nseg=0, stream=None):
    r, c = x.shape
    _check(lib().jetq_quant_mx32(_p(x), r, c, x.stride(0), _p(q_row), _p(e8_row), _p(q_col), _p(e8_col),
                                 ldq_col, _p(seg_offsets), nseg, _s(stream)), "jetq_quant_mx32")


def jetq_quant_act_1x128_pow2(x, q_row, e8_row, q_col, e8_col, ldq_col, seg_offsets=None, nseg=0, stream=None):
    r, c = x.shape
    _check(lib().jetq_quant_act_1x128_pow2(_p(x), r, c, x.stride(0), _p(q_row), _p(e8_row), _p(q_col), _p(e8_col),
                                           ldq_col, _p(seg_offsets), nseg, _s(stream)), "jetq_quant_act_1x128_pow2")


def jetq_quant_w_128x128_pow2(w, q, e8, qT=None, e8T=None, stream=None):
    d, c = w.shape
    _check(lib().jetq_quant_w_128x128_pow2(_p(w), d, c, w.stride(0), _p(q), _p(e8), _p(qT), _p(e8T), _s(stream)),
           "jetq_quant_w_128x128_pow2")


def jetq_requant_col_from_row(q_row, s_row, q_col, s_col, ldq_col, seg_offsets=None, nseg=0, stream=None):
    n, c = q_row.shape
    _check(lib().jetq_requant_col_from_row(_p(q_row), _p(s_row), n, c, _p(q_col), _p(s_col), ldq_col,
                                           _p(seg_offsets), nseg, _s(stream)), "jetq_requant_col_from_row")


SCALES_ROWGROUPS_1X128, SCALES_BLOCKS_128X128 = 0, 1


def jetq_dequant_bf16(q, s, layout, out, stream=None):
    rows, cols = q.shape
    _check(lib().jetq_dequant_bf16(_p(q), _p(s), rows, cols, layout, _p(out), out.stride(0), _s(stream)),
           "jetq_dequant_bf16")


def requant_col(q_row, s_row, seg_offsets=None, stream=None):
    """Column copy (q_col [c x cap], s_col [cap/128 x c], ldq_col) re-quantized from a row copy."""
    n, c = q_row.shape
    nseg = 0 if seg_offsets is None else seg_offsets.numel() - 1
    cap = jetq_colcopy_capacity(n, max(nseg, 1))
    q_col = torch.zeros((c, cap), dtype=torch.uint8, device=q_row.device)
    s_col = torch.zeros((max(cap, 128) // 128, c), dtype=torch.float32, device=q_row.device)
    jetq_requant_col_from_row(q_row, s_row, q_col, s_col, cap, seg_offsets, nseg, stream)
    return dict(q_col=q_col, s_col=s_col, ldq_col=cap)


def dequant_bf16(q, s, layout=SCALES_ROWGROUPS_1X128, stream=None):
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    jetq_dequant_bf16(q, s, layout, out, stream)
    return out


def _out_dtype(t):
    return OUT_BF16 if t.dtype == torch.bfloat16 else OUT_F32


def jetq_gemm_fprop(recipe, qx, sx, qw, sw, n, d, c, y, path=PATH_AUTO, stream=None):
    _check(lib().jetq_gemm_fprop(recipe, _p(qx), _p(sx), _p(qw), _p(sw), n, d, c, _p(y), _out_dtype(y),
                                 y.stride(0), path, _s(stream)), "jetq_gemm_fprop")


def jetq_decode_workspace_bytes(n, d, c):
    return int(lib().jetq_decode_workspace_bytes(n, d, c))


def jetq_gemm_fprop_ws(recipe, qx, sx, qw, sw, n, d, c, y, ws, path=PATH_AUTO, stream=None):
    _check(lib().jetq_gemm_fprop_ws(recipe, _p(qx), _p(sx), _p(qw), _p(sw), n, d, c, _p(y), _out_dtype(y),
                                    y.stride(0), None if ws is None else _p(ws),
                                    _bytes(ws), path, _s(stream)),
           "jetq_gemm_fprop_ws")


NOALLOC_SCRATCH_BYTES = 16 << 20  # JETQ_NOALLOC_SCRATCH_BYTES


def jetq_gemm_fprop_noalloc(qx, sx, qw, sw, n, d, c, y, stream=None):
    """Rollout FProp (128-block recipe, decode path) that allocates nothing: the
    split-K partial sums use a device array built into the library."""
    _check(lib().jetq_gemm_fprop_noalloc(_p(qx), _p(sx), _p(qw), _p(sw), n, d, c, _p(y), _out_dtype(y),
                                         y.stride(0), _s(stream)), "jetq_gemm_fprop_noalloc")


def jetq_gemm_dgrad(recipe, qdy, sdy, qwt, swt, n, d, c, dx, stream=None):
    _check(lib().jetq_gemm_dgrad(recipe, _p(qdy), _p(sdy), _p(qwt), _p(swt), n, d, c, _p(dx), _out_dtype(dx),
                                 dx.stride(0), _s(stream)), "jetq_gemm_dgrad")


def jetq_gemm_wgrad(recipe, qdyc, sdyc, qxc, sxc, k, ldk, d, c, dw, accumulate=False, stream=None):
    _check(lib().jetq_gemm_wgrad(recipe, _p(qdyc), _p(sdyc), _p(qxc), _p(sxc), k, ldk, d, c, _p(dw),
                                 dw.stride(0), 1 if accumulate else 0, _s(stream)), "jetq_gemm_wgrad")


def jetq_gemm_grouped(kind, recipe, a, sa, b, sb, m, n, k, ldk, seg_offsets, num_experts, out, accumulate=False,
                      stream=None):
    _check(lib().jetq_gemm_grouped(kind, recipe, _p(a), _p(sa), _p(b), _p(sb), m, n, k, ldk, _p(seg_offsets),
                                   num_experts, _p(out), _out_dtype(out), out.stride(-2), 1 if accumulate else 0,
                                   _s(stream)), "jetq_gemm_grouped")


def jetq_gemv_nvfp4(qw, sbw, sgw, x, y, stream=None):
    m, k = x.shape
    _check(lib().jetq_gemv_nvfp4(_p(qw), _p(sbw), _p(sgw), qw.shape[0], k, _p(x), m, x.stride(0), _p(y),
                                 _out_dtype(y), y.stride(0), _s(stream)), "jetq_gemv_nvfp4")


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def jetq_moe_nvfp4_workspace_bytes(m: int, num_experts: int, h: int, inter: int, topk: int) -> int:
    return int(lib().jetq_moe_nvfp4_workspace_bytes(m, num_experts, h, inter, topk))


def jetq_moe_nvfp4(x, router, topk, renorm, q13, sb13, sg13, q2, sb2, sg2, y, ids, weights, ws, stream=None):
    m, h = x.shape
    _check(lib().jetq_moe_nvfp4(x.data_ptr(), m, h, x.stride(0), router.data_ptr(), router.stride(0), router.shape[0],
                                topk, 1 if renorm else 0, q13.data_ptr(), sb13.data_ptr(), sg13.data_ptr(),
                                q13.shape[1] // 2, q2.data_ptr(), sb2.data_ptr(), sg2.data_ptr(), y.data_ptr(),
                                _out_dtype(y), y.stride(0), _p(ids), _p(weights), ws.data_ptr(), _bytes(ws),
                                _s(stream)), "jetq_moe_nvfp4")


def jetq_norm_fwd(kind, x, w, b, eps, y, mean, rstd, stream=None):
    n, c = x.shape
    _check(lib().jetq_norm_fwd(kind, _out_dtype(x), _p(x), n, c, x.stride(0), _p(w), _p(b), eps, _p(y), y.stride(0),
                               _p(mean), _p(rstd), _s(stream)), "jetq_norm_fwd")


def jetq_norm_bwd_workspace_bytes(dtype: int, n: int, c: int) -> int:
    return int(lib().jetq_norm_bwd_workspace_bytes(dtype, n, c))


def jetq_norm_bwd(kind, dy, x, w, mean, rstd, dx, dw, db, ws, stream=None):
    n, c = x.shape
    _check(lib().jetq_norm_bwd(kind, _out_dtype(x), _p(dy), dy.stride(0), _p(x), n, c, x.stride(0), _p(w), _p(mean),
                               _p(rstd), _p(dx), dx.stride(0), _p(dw), _p(db), _p(ws),
                               _bytes(ws), _s(stream)), "jetq_norm_bwd")


def jetq_linear_ce_workspace_bytes(n: int, v: int, c: int) -> int:
    return int(lib().jetq_linear_ce_workspace_bytes(n, v, c))


def jetq_linear_ce_fwd(x, w, target, scale, loss, lse, ws, stream=None):
    n, c = x.shape
    _check(lib().jetq_linear_ce_fwd(_p(x), n, c, x.stride(0), _p(w), w.shape[0], w.stride(0), _p(target), scale,
                                    _p(loss), _p(lse), _p(ws), _bytes(ws),
                                    _s(stream)), "jetq_linear_ce_fwd")


def jetq_linear_ce_bwd_workspace_bytes(n: int, v: int, c: int, smallest: bool = False) -> int:
    return int(lib().jetq_linear_ce_bwd_workspace_bytes(n, v, c, 1 if smallest else 0))


def jetq_linear_ce_bwd(x, w, target, scale, lse, dloss, dx, dw, accumulate, ws, stream=None):
    n, c = x.shape
    _check(lib().jetq_linear_ce_bwd(_p(x), n, c, x.stride(0), _p(w), w.shape[0], w.stride(0), _p(target), scale,
                                    _p(lse), _p(dloss), _p(dx), dx.stride(0), _p(dw), _out_dtype(dw), dw.stride(0),
                                    1 if accumulate else 0, _p(ws),
                                    _bytes(ws), _s(stream)),
           "jetq_linear_ce_bwd")


def jetq_linear_distill_workspace_bytes(n: int, v: int, c: int, k: int) -> int:
    return int(lib().jetq_linear_distill_workspace_bytes(n, v, c, k))


def jetq_linear_distill_fwd(x, w, ids, teacher, renorm, scale, loss, lse, logp, ws, stream=None):
    n, c = x.shape
    _check(lib().jetq_linear_distill_fwd(_p(x), n, c, x.stride(0), _p(w), w.shape[0], w.stride(0), _p(ids),
                                         ids.stride(0), _p(teacher), teacher.stride(0), ids.shape[1],
                                         1 if renorm else 0, scale, _p(loss), _p(lse), _p(logp), _p(ws), _bytes(ws),
                                         _s(stream)), "jetq_linear_distill_fwd")


def jetq_linear_distill_bwd_workspace_bytes(n: int, v: int, c: int, k: int, smallest: bool = False) -> int:
    return int(lib().jetq_linear_distill_bwd_workspace_bytes(n, v, c, k, 1 if smallest else 0))


def jetq_linear_distill_bwd(x, w, ids, teacher, renorm, scale, lse, logp, dloss, dx, dw, accumulate, ws, stream=None):
    n, c = x.shape
    _check(lib().jetq_linear_distill_bwd(_p(x), n, c, x.stride(0), _p(w), w.shape[0], w.stride(0), _p(ids),
                                         ids.stride(0), _p(teacher), teacher.stride(0), ids.shape[1],
                                         1 if renorm else 0, scale, _p(lse), _p(logp), _p(dloss), _p(dx),
                                         dx.stride(0), _p(dw), _out_dtype(dw), dw.stride(0), 1 if accumulate else 0,
                                         _p(ws), _bytes(ws), _s(stream)), "jetq_linear_distill_bwd")


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def jetq_policy_loss_workspace_bytes(n: int, nseg: int = 1) -> int:
    return int(lib().jetq_policy_loss_workspace_bytes(n, nseg))


def jetq_policy_loss_fwd(nll, nll_old, nll_ref, adv, adv_per_token, mask, seg_offsets, nseg, level, mean, scale,
                         clip_low, clip_high, clip_dual, kl, out, seg, ws, stream=None):
    _check(lib().jetq_policy_loss_fwd(nll.data_ptr(), nll_old.data_ptr(), _p(nll_ref), adv.data_ptr(), adv_per_token,
                                      _p(mask), nll.numel(), _p(seg_offsets), nseg, level, mean, scale, clip_low,
                                      clip_high, clip_dual, kl, out.data_ptr(), seg.data_ptr(), ws.data_ptr(),
                                      _bytes(ws), _s(stream)), "jetq_policy_loss_fwd")


def jetq_policy_loss_bwd(nll, nll_old, nll_ref, adv, adv_per_token, mask, seg_offsets, nseg, level, mean, scale,
                         clip_low, clip_high, clip_dual, kl, out, seg, dloss, dnll, stream=None):
    _check(lib().jetq_policy_loss_bwd(nll.data_ptr(), nll_old.data_ptr(), _p(nll_ref), adv.data_ptr(), adv_per_token,
                                      _p(mask), nll.numel(), _p(seg_offsets), nseg, level, mean, scale, clip_low,
                                      clip_high, clip_dual, kl, out.data_ptr(), seg.data_ptr(), _p(dloss),
                                      dnll.data_ptr(), _s(stream)), "jetq_policy_loss_bwd")


# ------------------------------------------------------------------ argument checks of the tensor helpers

def _want(t, name, dtype, shape=None, rows=False):
    """A CUDA tensor of `dtype` (and shape); rows: unit stride along the last axis, else dense."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is wanted")
    if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
        raise ValueError(f"{name}: {dtype} is wanted, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} is wanted, got {tuple(t.shape)}")
    if t.is_contiguous() and (not rows or t.dim() == 2):
        return
    if not rows:
        raise ValueError(f"{name}: a contiguous tensor is wanted")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name}: rows of consecutive elements are wanted, got strides {t.stride()}")


def _check_workspace(workspace, x):
    """A caller's workspace (None passes): consecutive bytes on x's device, all of them the kernels' to write."""
    if workspace is None:
        return
    if not isinstance(workspace, torch.Tensor) or workspace.device != x.device:
        raise ValueError(f"workspace: a tensor on {x.device} is wanted")
    if not workspace.is_contiguous():
        raise ValueError(f"workspace: consecutive elements are wanted, got strides {workspace.stride()}")


def _one_device(x, *tensors):
    """All tensors (None passes) on x's device, which is the current one: the launch goes to its stream."""
    at = x.get_device()
    if at != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {x.device}: make it the current device for the call")
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError(f"tensors on {x.device} and {t.device}: one device is wanted")


# ------------------------------------------------------------------ allocating helpers

def quant_act(x, row=True, col=True, seg_offsets=None, stream=None):
    """BF16 [n x c] -> dict(q_row, s_row, q_col, s_col, ldq_col) (absent copies are None)."""
    n, c = x.shape
    dev = x.device
    nseg = 0 if seg_offsets is None else seg_offsets.numel() - 1
    cap = jetq_colcopy_capacity(n, max(nseg, 1))
    out = dict(q_row=None, s_row=None, q_col=None, s_col=None, ldq_col=cap)
    if row:
        out["q_row"] = torch.empty((n, c), dtype=torch.uint8, device=dev)
        out["s_row"] = torch.empty((c // 128, n), dtype=torch.float32, device=dev)
    if col:
        out["q_col"] = torch.empty((c, cap), dtype=torch.uint8, device=dev)
        out["s_col"] = torch.empty((max(cap, 128) // 128, c), dtype=torch.float32, device=dev)
    jetq_quant_act_1x128(x, out["q_row"], out["s_row"], out["q_col"], out["s_col"], cap, seg_offsets, nseg, stream)
    return out


def _act_copies(n, c, dev, row, col, seg_offsets):
    nseg = 0 if seg_offsets is None else seg_offsets.numel() - 1
    cap = jetq_colcopy_capacity(n, max(nseg, 1))
    out = dict(q_row=None, s_row=None, q_col=None, s_col=None, ldq_col=cap)
    if row:
        out["q_row"] = torch.empty((n, c), dtype=torch.uint8, device=dev)
        out["s_row"] = torch.empty((c // 128, n), dtype=torch.float32, device=dev)
    if col:
        out["q_col"] = torch.empty((c, cap), dtype=torch.uint8, device=dev)
        out["s_col"] = torch.empty((max(cap, 128) // 128, c), dtype=torch.float32, device=dev)
    return out, nseg


def quant_act_rmsnorm(x, w, eps=1e-6, row=True, col=True, seg_offsets=None, stream=None):
    """1x128 copies of RMSNorm(x) * w (BF16, not stored): the quant_act dict plus rstd [n]."""
    n, c = x.shape
    out, nseg = _act_copies(n, c, x.device, row, col, seg_offsets)
    out["rstd"] = torch.empty(n, dtype=torch.float32, device=x.device)
    jetq_quant_act_1x128_rmsnorm(x, w, eps, out["rstd"], out["q_row"], out["s_row"], out["q_col"], out["s_col"],
                                 out["ldq_col"], seg_offsets, nseg, stream)
    return out


def quant_act_swiglu(gate, up, row=True, col=True, seg_offsets=None, stream=None):
    """1x128 copies of silu(gate) * up (BF16, not stored), as the quant_act dict."""
    n, c = gate.shape
    out, nseg = _act_copies(n, c, gate.device, row, col, seg_offsets)
    jetq_quant_act_1x128_swiglu(gate, up, out["q_row"], out["s_row"], out["q_col"], out["s_col"], out["ldq_col"],
                                seg_offsets, nseg, stream)
    return out


def quant_nvfp4(x, scope_amax=None, stream=None):
    """NVFP4 copy of BF16 x: dict(q [r x c/2] u8, sb [r x c/16] u8, sg [r] or [1] f32).
    scope_amax: a device float tensor (tensor scope) or None (one scope per row)."""
    r, c = x.shape
    dev = x.device
    out = dict(q=torch.empty((r, c // 2), dtype=torch.uint8, device=dev),
               sb=torch.empty((r, c // 16), dtype=torch.uint8, device=dev),
               sg=torch.empty(r if scope_amax is None else 1, dtype=torch.float32, device=dev))
    jetq_quant_nvfp4(x, out["q"], out["sb"], out["sg"], scope_amax, stream)
    return out


def amax_bf16(*tensors, stream=None):
    """max |x| over one or more BF16 tensors, as a device float tensor of one element."""
    a = torch.zeros(1, dtype=torch.float32, device=tensors[0].device)
    for t in tensors:
        jetq_amax_bf16(t, a, stream)
    return a


def dequant_nvfp4_bf16(q, sb, sg, stream=None):
    """BF16 values of an NVFP4 copy (per-row scope when sg has one entry per row)."""
    r = q.shape[0]
    out = torch.empty((r, q.shape[1] * 2), dtype=torch.bfloat16, device=q.device)
    jetq_dequant_nvfp4_bf16(q, sb, sg, sg.numel() > 1, out, stream)
    return out


def nvfp4_atoms(sb, k, stream=None):
    """Scale atoms (the block-scaled FP4 MMA's layout) of row-major NVFP4 block scales sb [rows x k/16]."""
    rows = sb.shape[0]
    atoms = torch.empty(jetq_nvfp4_atom_bytes(rows, k), dtype=torch.uint8, device=sb.device)
    jetq_nvfp4_scale_atoms(sb, rows, k, atoms, stream)
    return atoms


def nvfp4_fprop(a, b, k, out_dtype=torch.float32, stream=None):
    """NVFP4 FProp of two quant_nvfp4 dicts (A: activations, B: weight), each with 'atoms' added."""
    m, n = a["q"].shape[0], b["q"].shape[0]
    y = torch.empty((m, n), dtype=out_dtype, device=a["q"].device)
    jetq_gemm_nvfp4(a["q"], a["atoms"], a["sg"], a["sg"].numel() > 1, b["q"], b["atoms"], b["sg"], m, n, k, y,
                    stream)
    return y


def quant_weight(w, transposed=True, stream=None):
    """BF16 [d x c] -> (q [d x c], s [d/128 x c/128], qT [c x d] | None, sT | None)."""
    d, c = w.shape
    dev = w.device
    q = torch.empty((d, c), dtype=torch.uint8, device=dev)
    s = torch.empty((d // 128, c // 128), dtype=torch.float32, device=dev)
    qT = torch.empty((c, d), dtype=torch.uint8, device=dev) if transposed else None
    sT = torch.empty((c // 128, d // 128), dtype=torch.float32, device=dev) if transposed else None
    jetq_quant_w_128x128(w, q, s, qT, sT, stream)
    return q, s, qT, sT


def quant_mx(x, row=True, col=True, seg_offsets=None, stream=None):
    """MXFP8 copies: dict(q_row, e8_row, q_col, e8_col, ldq_col); scales in the atom layout."""
    r, c = x.shape
    dev = x.device
    nseg = 0 if seg_offsets is None else seg_offsets.numel() - 1
    cap = jetq_colcopy_capacity(r, max(nseg, 1))
    out = dict(q_row=None, e8_row=None, q_col=None, e8_col=None, ldq_col=cap)
    if row:
        out["q_row"] = torch.empty((r, c), dtype=torch.uint8, device=dev)
        out["e8_row"] = torch.zeros(jetq_mx_scale_bytes(r, c), dtype=torch.uint8, device=dev)
    if col:
        out["q_col"] = torch.empty((c, cap), dtype=torch.uint8, device=dev)
        out["e8_col"] = torch.zeros(jetq_mx_scale_bytes(c, cap), dtype=torch.uint8, device=dev)
    jetq_quant_mx32(x, out["q_row"], out["e8_row"], out["q_col"], out["e8_col"], cap, seg_offsets, nseg, stream)
    return out


def quant_act_pow2(x, row=True, col=True, seg_offsets=None, stream=None):
    """Power-of-two 1x128 / 128x1 copies: dict(q_row, e8_row, q_col, e8_col, ldq_col), MX atom layout."""
    r, c = x.shape
    dev = x.device
    nseg = 0 if seg_offsets is None else seg_offsets.numel() - 1
    cap = jetq_colcopy_capacity(r, max(nseg, 1))
    out = dict(q_row=None, e8_row=None, q_col=None, e8_col=None, ldq_col=cap)
    if row:
        out["q_row"] = torch.empty((r, c), dtype=torch.uint8, device=dev)
        out["e8_row"] = torch.zeros(jetq_mx_scale_bytes(r, c), dtype=torch.uint8, device=dev)
    if col:
        out["q_col"] = torch.empty((c, cap), dtype=torch.uint8, device=dev)
        out["e8_col"] = torch.zeros(jetq_mx_scale_bytes(c, cap), dtype=torch.uint8, device=dev)
    jetq_quant_act_1x128_pow2(x, out["q_row"], out["e8_row"], out["q_col"], out["e8_col"], cap, seg_offsets, nseg,
                              stream)
    return out


def quant_weight_pow2(w, transposed=True, stream=None):
    """Power-of-two 128x128 blocks: (q [d x c], e8 atoms (d, c), qT [c x d] | None, e8T atoms (c, d) | None)."""
    d, c = w.shape
    dev = w.device
    q = torch.empty((d, c), dtype=torch.uint8, device=dev)
    e8 = torch.zeros(jetq_mx_scale_bytes(d, c), dtype=torch.uint8, device=dev)
    qT = torch.empty((c, d), dtype=torch.uint8, device=dev) if transposed else None
    e8T = torch.zeros(jetq_mx_scale_bytes(c, d), dtype=torch.uint8, device=dev) if transposed else None
    jetq_quant_w_128x128_pow2(w, q, e8, qT, e8T, stream)
    return q, e8, qT, e8T


def fprop(qx, sx, qw, sw, out_dtype=torch.float32, path=PATH_AUTO, recipe=RECIPE_BLOCK128, stream=None,
          workspace=None):
    """Y = X W^T.  Rollout-sized calls that can spread a weight band over several
    SMs get a workspace (the caller's, if large enough, else a fresh one)."""
    n, c = qx.shape
    d = qw.shape[0]
    _check_workspace(workspace, qx)
    y = torch.empty((n, d), dtype=out_dtype, device=qx.device)
    wsb = jetq_decode_workspace_bytes(n, d, c) if recipe == RECIPE_BLOCK128 and path != PATH_TRAIN else 0
    if wsb:
        if workspace is None or workspace.numel() * workspace.element_size() < wsb:
            workspace = torch.empty(wsb, dtype=torch.uint8, device=qx.device)
        jetq_gemm_fprop_ws(recipe, qx, sx, qw, sw, n, d, c, y, workspace, path, stream)
    else:
        jetq_gemm_fprop(recipe, qx, sx, qw, sw, n, d, c, y, path, stream)
    return y


def dgrad(qdy, sdy, qwt, swt, out_dtype=torch.float32, recipe=RECIPE_BLOCK128, stream=None):
    n, d = qdy.shape
    c = qwt.shape[0]
    dx = torch.empty((n, c), dtype=out_dtype, device=qdy.device)
    jetq_gemm_dgrad(recipe, qdy, sdy, qwt, swt, n, d, c, dx, stream)
    return dx


def wgrad(qdyc, sdyc, qxc, sxc, k, dw=None, accumulate=False, recipe=RECIPE_BLOCK128, stream=None):
    d, ldk = qdyc.shape
    c = qxc.shape[0]
    if dw is None:
        dw = torch.empty((d, c), dtype=torch.float32, device=qdyc.device)
    jetq_gemm_wgrad(recipe, qdyc, sdyc, qxc, sxc, k, ldk, d, c, dw, accumulate, stream)
    return dw


def grouped(kind, a, sa, b, sb, seg_offsets, n, k, out_dtype=torch.float32, recipe=RECIPE_BLOCK128, out=None,
            accumulate=False, stream=None):
    """Per-expert GEMMs over routed rows (see jetq_gemm_grouped).

    FPROP/DGRAD: a [m x k] routed row copy, b stacked [E*n x k] (or [E, n, k]); returns [m x n].
    WGRAD: a, b column copies [m x ldk], [n x ldk]; k = column-copy length; returns [E x m x n] FP32.
    """
    E = seg_offsets.numel() - 1
    m, ldk = a.shape[0], a.shape[1]
    if out is None:
        if kind == GEMM_WGRAD:
            out = torch.empty((E, m, n), dtype=torch.float32, device=a.device)
        else:
            out = torch.empty((m, n), dtype=out_dtype, device=a.device)
    jetq_gemm_grouped(kind, recipe, a, sa, b, sb, m, n, k, ldk, seg_offsets, E, out, accumulate, stream)
    return out


# The helpers below allocate on the stream that they launch on (workspaces are
# released when they return, and their memory must not be reused on another
# stream before the kernels are done with it).

def gemv_nvfp4(x, b, out_dtype=torch.float32, stream=None):
    """Few-token product of BF16 x [m x k], m <= 16, with a quant_nvfp4 dict b of a weight
    [n x k] (tensor scope; see jetq_gemv_nvfp4) -> [m x n]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gemv_nvfp4(x, b, out_dtype)
    q, sb, sg = b["q"], b["sb"], b["sg"]
    _want(x, "x", torch.bfloat16, rows=True)
    (m, k), n = x.shape, q.shape[0]
    _want(q, "q", torch.uint8, (n, k // 2))
    _want(sb, "sb", torch.uint8, (n, k // 16))
    _want(sg, "sg", torch.float32, (1,))
    y = torch.empty((m, n), dtype=out_dtype, device=x.device)
    jetq_gemv_nvfp4(q, sb, sg, x, y)
    return y


def quant_nvfp4_experts(w, stream=None):
    """NVFP4 copies of stacked expert weights, BF16 w [e x r x c] (rows of consecutive elements), a tensor scope each:
    dict(q [e x r x c/2] u8, sb [e x r x c/16] u8, sg [e] f32), as moe_nvfp4 takes them."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quant_nvfp4_experts(w)
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w: a tensor [experts x rows x columns] is wanted")
    e, r, c = w.shape
    if e > 0:
        _want(w[0], "an expert's weight", torch.bfloat16, rows=True)  # the others are laid out alike
        _one_device(w)
    out = dict(q=torch.empty((e, r, c // 2), dtype=torch.uint8, device=w.device),
               sb=torch.empty((e, r, c // 16), dtype=torch.uint8, device=w.device),
               sg=torch.empty(e, dtype=torch.float32, device=w.device))
    for i in range(e):
        one = _row_stride(w[i])
        jetq_quant_nvfp4(one, out["q"][i], out["sb"][i], out["sg"][i:i + 1], amax_bf16(one))
    return out


def moe_nvfp4(x, router, w13, w2, topk, renorm=True, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """Mixture-of-experts layer for up to 16 tokens (see jetq_moe_nvfp4): BF16 x [m x h], router [e x h], NVFP4
    dicts (as quant_nvfp4_experts makes them) w13 of [e x 2i x h], gate rows before up rows, and w2 of [e x h x i]
    -> (y [m x h], ids int64 [m x topk], p [m x topk])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_nvfp4(x, router, w13, w2, topk, renorm, out_dtype, workspace)
    _want(x, "x", torch.bfloat16, rows=True)
    _want(router, "router", torch.bfloat16, rows=True)
    (m, h), e = x.shape, router.shape[0]
    if router.shape[1] != h:
        raise ValueError(f"x and router: widths {h} and {router.shape[1]}")
    q13, sb13, sg13, q2, sb2, sg2 = w13["q"], w13["sb"], w13["sg"], w2["q"], w2["sb"], w2["sg"]
    i = q2.shape[-1] * 2
    _want(q13, "w13['q']", torch.uint8, (e, 2 * i, h // 2))
    _want(sb13, "w13['sb']", torch.uint8, (e, 2 * i, h // 16))
    _want(sg13, "w13['sg']", torch.float32, (e,))
    _want(q2, "w2['q']", torch.uint8, (e, h, i // 2))
    _want(sb2, "w2['sb']", torch.uint8, (e, h, i // 16))
    _want(sg2, "w2['sg']", torch.float32, (e,))
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype: {out_dtype} is neither BF16 nor FP32")
    _one_device(x, router, q13, sb13, sg13, q2, sb2, sg2)
    _check_workspace(workspace, x)
    y = torch.empty((m, h), dtype=out_dtype, device=x.device)
    ids = torch.empty((m, topk), dtype=torch.int64, device=x.device)
    p = torch.empty((m, topk), dtype=torch.float32, device=x.device)
    need = jetq_moe_nvfp4_workspace_bytes(m, e, h, i, topk)
    if workspace is None or _bytes(workspace) < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    jetq_moe_nvfp4(_row_stride(x), _row_stride(router), topk, renorm, q13, sb13, sg13, q2, sb2, sg2, y, ids, p,
                   workspace)
    return y, ids, p


_NORM_DTYPES = (torch.bfloat16, torch.float32)


def _norm_rows(x, n, c):
    """An uninitialized tensor like x whose rows are 16-byte aligned."""
    pad = -c % (8 if x.dtype is torch.bfloat16 else 4)
    if pad == 0:
        return torch.empty((n, c), dtype=x.dtype, device=x.device)
    return torch.empty_strided((n, c), (c + pad, 1), dtype=x.dtype, device=x.device)


def _aligned_rows(x):
    """x as the norm kernels take it: itself, or a padded copy where its rows are not 16-byte aligned."""
    n, c = x.shape
    ld = x.stride(0)
    if ld >= c and ld % (8 if x.dtype is torch.bfloat16 else 4) == 0 and x.data_ptr() % 16 == 0:
        return x
    return _norm_rows(x, n, c).copy_(x)


def norm_fwd(x, w=None, b=None, eps=1e-5, kind=NORM_LAYER, stream=None):
    """Layer norm or RMS norm of BF16 or FP32 rows x [n x c] (see jetq_norm_fwd) ->
    (y, mean [n] (None for RMS), rstd [n]).  The kernels read rows that start on 16 bytes: x in
    other rows (a dense one of odd width, a view off the boundary) is copied to padded ones
    first, and y's rows are padded where the width asks for it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return norm_fwd(x, w, b, eps, kind)
    _want(x, "x", _NORM_DTYPES, rows=True)
    n, c = x.shape
    if w is not None:
        _want(w, "w", x.dtype, (c,))
    if b is not None:
        _want(b, "b", x.dtype, (c,))
    x = _aligned_rows(x)
    y = _norm_rows(x, n, c)
    rstd = torch.empty(n, dtype=torch.float32, device=x.device)
    mean = torch.empty(n, dtype=torch.float32, device=x.device) if kind == NORM_LAYER else None
    jetq_norm_fwd(kind, x, w, b, eps, y, mean, rstd)
    return y, mean, rstd


def norm_bwd(dy, x, w, mean, rstd, kind=NORM_LAYER, bias=False, workspace=None, stream=None):
    """Backward pass of norm_fwd (see jetq_norm_bwd) -> (dx, dw FP32 [c], db FP32 [c] or None).
    dy and x are copied, and dx is padded, as norm_fwd does it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return norm_bwd(dy, x, w, mean, rstd, kind, bias, workspace)
    _want(x, "x", _NORM_DTYPES, rows=True)
    n, c = x.shape
    _want(dy, "dy", x.dtype, (n, c), rows=True)
    if w is not None:
        _want(w, "w", x.dtype, (c,))
    _want(rstd, "rstd", torch.float32, (n,))
    if kind == NORM_LAYER:
        _want(mean, "mean", torch.float32, (n,))
    _check_workspace(workspace, x)
    dy, x = _aligned_rows(dy), _aligned_rows(x)
    dx = _norm_rows(x, n, c)
    dw = torch.empty(c, dtype=torch.float32, device=x.device)
    db = torch.empty(c, dtype=torch.float32, device=x.device) if bias else None
    if workspace is None:
        workspace = torch.empty(jetq_norm_bwd_workspace_bytes(_out_dtype(x), n, c), dtype=torch.uint8,
                                device=x.device)
    jetq_norm_bwd(kind, dy, x, w, mean if kind == NORM_LAYER else None, rstd, dx, dw, db, workspace)
    return dx, dw, db


def _check_head(x, w, target):
    _want(x, "x", torch.bfloat16, rows=True)
    _want(w, "w", torch.bfloat16, rows=True)
    _want(target, "target", torch.int64, (x.shape[0],))
    if x.shape[1] != w.shape[1]:
        raise ValueError(f"x and w: widths {x.shape[1]} and {w.shape[1]}")


def linear_ce(x, w, target, scale=1.0, workspace=None, stream=None):
    """Token losses of a linear head (see jetq_linear_ce_fwd): BF16 x [n x c], w [v x c], int64
    target [n] (outside [0, v): no loss) -> (loss [n], lse [n])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_ce(x, w, target, scale, workspace)
    _check_head(x, w, target)
    _check_workspace(workspace, x)
    (n, c), v = x.shape, w.shape[0]
    loss = torch.empty(n, dtype=torch.float32, device=x.device)
    lse = torch.empty(n, dtype=torch.float32, device=x.device)
    need = jetq_linear_ce_workspace_bytes(n, v, c)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    jetq_linear_ce_fwd(x, w, target, scale, loss, lse, workspace)
    return loss, lse


def linear_ce_bwd(x, w, target, lse, dloss, scale=1.0, dw_dtype=torch.float32, dw=None, accumulate=False,
                  workspace=None, stream=None):
    """Gradient of linear_ce (see jetq_linear_ce_bwd) -> (dx BF16 [n x c], dw [v x c]).  A workspace
    that the caller gives is used as it is: its size decides the vocabulary's pieces."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_ce_bwd(x, w, target, lse, dloss, scale, dw_dtype, dw, accumulate, workspace)
    _check_head(x, w, target)
    _check_workspace(workspace, x)
    (n, c), v = x.shape, w.shape[0]
    _want(lse, "lse", torch.float32, (n,))
    _want(dloss, "dloss", torch.float32, (n,))
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs a dw to add into")
        dw = torch.empty((v, c), dtype=dw_dtype, device=x.device)
    _want(dw, "dw", (torch.float32, torch.bfloat16), (v, c), rows=True)
    dx = torch.empty((n, c), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(jetq_linear_ce_bwd_workspace_bytes(n, v, c), dtype=torch.uint8, device=x.device)
    jetq_linear_ce_bwd(x, w, target, scale, lse, dloss, dx, dw, accumulate, workspace)
    return dx, dw


def _check_distill(x, w, ids, teacher):
    _want(x, "x", torch.bfloat16, rows=True)
    _want(w, "w", torch.bfloat16, rows=True)
    n = x.shape[0]
    _want(ids, "ids", torch.int64, rows=True)
    _want(teacher, "teacher", torch.float32, ids.shape, rows=True)
    if ids.shape[0] != n or not 1 <= ids.shape[1] <= 256:
        raise ValueError(f"ids: {n} rows of 1 to 256 entries are wanted, got shape {tuple(ids.shape)}")
    if x.shape[1] != w.shape[1]:
        raise ValueError(f"x and w: widths {x.shape[1]} and {w.shape[1]}")
    _one_device(x, w, ids, teacher)


def _row_stride(t):
    """t with a row stride that covers its rows (a single row may carry any)."""
    return t if t.shape[0] > 1 or t.stride(0) >= t.shape[1] else t.reshape(-1).as_strided(t.shape, (t.shape[1], 1))


def linear_distill(x, w, ids, teacher, scale=1.0, renorm=True, workspace=None, stream=None):
    """Distillation losses of a linear head from a teacher's top logits (see jetq_linear_distill_fwd): BF16 x
    [n x c], w [v x c], int64 ids [n x k] (outside [0, v): nothing listed), FP32 teacher [n x k] (logits with
    renorm, else log-probabilities) -> (loss [n], lse [n], logp [n x k])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_distill(x, w, ids, teacher, scale, renorm, workspace)
    _check_distill(x, w, ids, teacher)
    _check_workspace(workspace, x)
    (n, c), v, k = x.shape, w.shape[0], ids.shape[1]
    loss = torch.empty(n, dtype=torch.float32, device=x.device)
    lse = torch.empty(n, dtype=torch.float32, device=x.device)
    logp = torch.empty((n, k), dtype=torch.float32, device=x.device)
    need = jetq_linear_distill_workspace_bytes(n, v, c, k)
    if workspace is None or _bytes(workspace) < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    jetq_linear_distill_fwd(_row_stride(x), _row_stride(w), _row_stride(ids), _row_stride(teacher), renorm, scale,
                            loss, lse, logp, workspace)
    return loss, lse, logp


def linear_distill_bwd(x, w, ids, teacher, lse, logp, dloss, scale=1.0, renorm=True, dw_dtype=torch.float32, dw=None,
                       accumulate=False, workspace=None, stream=None):
    """Gradient of linear_distill (see jetq_linear_distill_bwd) -> (dx BF16 [n x c], dw [v x c]).  A workspace that
    the caller gives is used as it is: its size decides the vocabulary's pieces."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_distill_bwd(x, w, ids, teacher, lse, logp, dloss, scale, renorm, dw_dtype, dw, accumulate,
                                      workspace)
    _check_distill(x, w, ids, teacher)
    _check_workspace(workspace, x)
    (n, c), v, k = x.shape, w.shape[0], ids.shape[1]
    _want(lse, "lse", torch.float32, (n,))
    _want(logp, "logp", torch.float32, (n, k))
    _want(dloss, "dloss", torch.float32, (n,))
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs a dw to add into")
        dw = torch.empty((v, c), dtype=dw_dtype, device=x.device)
    _want(dw, "dw", (torch.float32, torch.bfloat16), (v, c), rows=True)
    _one_device(x, lse, logp, dloss, dw)
    dx = torch.empty((n, c), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(jetq_linear_distill_bwd_workspace_bytes(n, v, c, k), dtype=torch.uint8,
                                device=x.device)
    jetq_linear_distill_bwd(_row_stride(x), _row_stride(w), _row_stride(ids), _row_stride(teacher), renorm, scale,
                            lse, logp, dloss, dx, dw, accumulate, workspace)
    return dx, dw


def _policy_args(nll, nll_old, adv, seg_offsets, nll_ref, mask, workspace=None, out=None, seg=None, dloss=None):
    """Checks of the policy loss's tensors -> the number of sequences."""
    f32, shape = torch.float32, nll.shape
    _want(nll, "nll", f32)
    if len(shape) != 1:
        raise ValueError(f"nll: one axis is wanted, got shape {tuple(shape)}")
    _want(nll_old, "nll_old", f32, shape)
    nseg = 1
    if seg_offsets is not None:
        _want(seg_offsets, "seg_offsets", torch.int64)
        nseg = seg_offsets.numel() - 1
        if seg_offsets.dim() != 1 or nseg < 1:
            raise ValueError(f"seg_offsets: at least two on one axis, got shape {tuple(seg_offsets.shape)}")
    _want(adv, "adv", f32)
    if adv.shape != shape and adv.shape != (nseg,):
        raise ValueError(f"adv: one for each of {shape[0]} tokens or of {nseg} sequences, got shape "
                         f"{tuple(adv.shape)}")
    if nll_ref is not None:
        _want(nll_ref, "nll_ref", f32, shape)
    if mask is not None:
        _want(mask, "mask", (torch.bool, torch.uint8), shape)
    if out is not None:
        _want(out, "out", f32, (6,))
        _want(seg, "seg", f32, (nseg, 2))
    if dloss is not None:
        _want(dloss, "dloss", f32)
        if dloss.numel() != 1:
            raise ValueError(f"dloss: one value is wanted, got shape {tuple(dloss.shape)}")
    _one_device(nll, nll_old, adv, seg_offsets, nll_ref, mask, out, seg, dloss)
    _check_workspace(workspace, nll)
    return nseg


def _adv_per_token(adv, n, nseg, adv_per_token):
    """Where there are as many tokens as sequences the shape does not tell: per sequence unless it is said."""
    if adv_per_token is None:
        return adv.shape[0] != nseg
    if adv.shape[0] != (n if adv_per_token else nseg):
        raise ValueError(f"adv: {n if adv_per_token else nseg} are wanted, got {adv.shape[0]}")
    return bool(adv_per_token)


def policy_loss(nll, nll_old, adv, seg_offsets=None, nll_ref=None, mask=None, clip_low=0.2, clip_high=0.2,
                clip_dual=0.0, kl=0.0, level=POLICY_TOKEN, mean=POLICY_MEAN_TOKENS, scale=1.0, adv_per_token=None,
                workspace=None, stream=None):
    """Clipped policy-gradient loss of packed sequences (see jetq_policy_loss_fwd): FP32 token losses nll, nll_old
    and nll_ref [n], advantages adv of the tokens [n] or of the sequences [nseg] (where both have the same number,
    adv_per_token tells; None: of the sequences), int64 seg_offsets [nseg + 1], mask bool or uint8 [n] ->
    (out [6]: loss, its policy part, its mean KL, clipped tokens, counted tokens, counted sequences;
    seg [nseg x 2] for the backward pass)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return policy_loss(nll, nll_old, adv, seg_offsets, nll_ref, mask, clip_low, clip_high, clip_dual, kl,
                               level, mean, scale, adv_per_token, workspace)
    nseg = _policy_args(nll, nll_old, adv, seg_offsets, nll_ref, mask, workspace)
    n = nll.shape[0]
    per_token = _adv_per_token(adv, n, nseg, adv_per_token)
    out = torch.empty(6, dtype=torch.float32, device=nll.device)
    seg = torch.empty((nseg, 2), dtype=torch.float32, device=nll.device)
    need = jetq_policy_loss_workspace_bytes(n, nseg)
    if workspace is None or _bytes(workspace) < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=nll.device)
    jetq_policy_loss_fwd(nll, nll_old, nll_ref, adv, per_token, mask, seg_offsets, nseg, level, mean, scale, clip_low,
                         clip_high, clip_dual, kl, out, seg, workspace)
    return out, seg


def policy_loss_bwd(nll, nll_old, adv, out, seg, seg_offsets=None, nll_ref=None, mask=None, clip_low=0.2,
                    clip_high=0.2, clip_dual=0.0, kl=0.0, level=POLICY_TOKEN, mean=POLICY_MEAN_TOKENS, scale=1.0,
                    adv_per_token=None, dloss=None, stream=None):
    """Gradient of policy_loss's out[0] (times dloss [1], where given) with respect to nll (see
    jetq_policy_loss_bwd) -> dnll [n], which linear_ce_bwd takes as its dloss."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return policy_loss_bwd(nll, nll_old, adv, out, seg, seg_offsets, nll_ref, mask, clip_low, clip_high,
                                   clip_dual, kl, level, mean, scale, adv_per_token, dloss)
    if out is None or seg is None:
        raise ValueError("out and seg: those of the forward call are wanted")
    nseg = _policy_args(nll, nll_old, adv, seg_offsets, nll_ref, mask, None, out, seg, dloss)
    per_token = _adv_per_token(adv, nll.shape[0], nseg, adv_per_token)
    dnll = torch.empty_like(nll)
    jetq_policy_loss_bwd(nll, nll_old, nll_ref, adv, per_token, mask, seg_offsets, nseg, level, mean, scale, clip_low,
                         clip_high, clip_dual, kl, out, seg, dloss, dnll)
    return dnll
