"""The operators around the product (include/tgemm_ops.h) on torch tensors:
``linear``, ``gemm_tn``, ``act_grad`` and ``linear_cross_entropy``.

As in ``_binding`` everything here marshals arguments; all arithmetic runs in
the HIP kernels, on torch's current stream of the operands' device. Workspaces
come from torch's allocator on that stream. ``linear`` and
``linear_cross_entropy`` take part in autograd (first derivatives, backward
mode; operands with forward-mode tangents are refused, and so are torch.func's
transforms).
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

from ._binding import (_DTYPE, _LAYOUT, TGEMM_B_NxK, TGEMM_BF16, TGEMM_F16, TGEMM_F32,
                       TGEMM_OK, TgemmError, _code, load)

TGEMM_ACT_SILU = 2
TGEMM_ACT_GELU = 3
TGEMM_ACT_GELU_TANH = 4
TGEMM_REDUCE_NONE = 0
TGEMM_REDUCE_SUM = 1
TGEMM_REDUCE_MEAN = 2

_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_REDUCE = {"none": 0, "sum": 1, "mean": 2}
_I64, _INT, _P, _F = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
_lib = None


def _ops():
    """libtgemm.so with the operators' signatures."""
    global _lib
    if _lib is None:
        lib = load()
        lin = [_I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _INT, _P, _INT, _INT, _P, _I64, _INT, _P, _I64, _P, _I64,
               _F, _P, _I64, _P]
        sigs = {
            "tgemm_linear": (_INT, lin),
            "tgemm_linear_config": (_INT, lin + [_INT, _INT, _INT]),
            "tgemm_linear_workspace": (_I64, [_I64, _I64, _I64, _INT, _I64, _I64, _INT, _INT, _I64]),
            "tgemm_linear_config_workspace": (_I64, [_I64, _I64, _I64, _INT, _I64, _I64, _INT, _INT, _I64, _INT, _INT,
                                                     _INT]),
            "tgemm_tn": (_INT, [_I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _INT, _P, _I64, _F, _INT, _P, _I64, _P,
                                _INT, _INT, _INT]),
            "tgemm_tn_workspace": (_I64, [_I64, _I64, _I64, _INT, _I64, _I64, _INT, _I64, _INT, _INT, _INT]),
            "tgemm_act_grad": (_INT, [_I64, _I64, _INT, _P, _I64, _INT, _P, _I64, _P, _I64, _INT, _P, _P, _I64, _P]),
            "tgemm_act_grad_workspace": (_I64, [_I64, _I64]),
            "tgemm_act_grad_f32": (_INT, [_I64, _I64, _INT, _P, _I64, _INT, _P, _I64, _P, _I64, _P, _INT, _P, _P, _I64, _P]),
            "tgemm_act_grad_f32_workspace": (_I64, [_I64, _I64]),
            "tgemm_linear_grad": (_INT, [_I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _INT, _INT, _P, _I64, _P, _I64, _P,
                                         _I64, _P, _I64, _INT, _P, _P, _I64, _P]),
            "tgemm_linear_grad_workspace": (_I64, [_I64, _I64, _I64, _INT, _I64, _I64, _INT, _INT, _I64, _I64, _I64]),
            "tgemm_xent": (_INT, [_I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _P, _I64, _INT, _P, _P, _P, _P, _P, _I64,
                                  _P]),
            "tgemm_xent_workspace": (_I64, [_I64, _I64, _I64, _INT, _I64, _I64]),
            "tgemm_xent_grad": (_INT, [_I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _P, _I64, _P, _P, _INT, _P, _P, _P,
                                       _I64, _P, _I64, _P, _I64, _P]),
            "tgemm_xent_grad_workspace": (_I64, [_I64, _I64, _I64, _INT, _I64, _I64, _I64, _I64]),
            "tgemm_xent_both": (_INT, [_I64, _I64, _I64, _INT, _P, _I64, _P, _I64, _P, _I64, _INT, _P, _P, _P, _P, _P, _I64,
                                       _P, _I64, _P, _I64, _P]),
            "tgemm_xent_both_workspace": (_I64, [_I64, _I64, _I64, _INT, _I64, _I64, _I64, _I64]),
            "tgemm_scale": (_INT, [_INT, _I64, _P, _I64, _P, _P, _P]),
        }
        for name in ("tgemm_linear_grad", "tgemm_linear_grad_workspace"):
            sigs[name.replace("_grad", "_grad_f32")] = sigs[name]
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


# --------------------------------------------------------------- raw calls --
# Pointers are integers (device addresses) or None; each returns the status.

def tgemm_linear(M, N, K, type, X, ldx, W, ldw, w_layout, bias=None, bias_type="f32", act="none", residual=None, ldr=0,
                 y_type=None, Y=None, ldy=0, pre=None, ldpre=0, alpha=1.0, workspace=None, workspace_bytes=0,
                 stream=None, tile_m=0, splits=0, k_step=0) -> int:
    t = _code(_DTYPE, type)
    return int(_ops().tgemm_linear_config(
        M, N, K, t, X, ldx, W, ldw, _LAYOUT.get(w_layout, w_layout), bias, _code(_DTYPE, bias_type), _code(_ACTS, act),
        residual, ldr, t if y_type is None else _code(_DTYPE, y_type), Y, ldy, pre, ldpre, float(alpha), workspace,
        workspace_bytes, stream, int(tile_m), int(k_step), int(splits)))


def tgemm_linear_workspace(M, N, K, type, ldx, ldw, w_layout, y_type, ldy, tile_m=0, splits=0, k_step=0) -> int:
    """Bytes, or a negative status."""
    return int(_ops().tgemm_linear_config_workspace(M, N, K, _code(_DTYPE, type), ldx, ldw,
                                                    _LAYOUT.get(w_layout, w_layout), _code(_DTYPE, y_type), ldy,
                                                    int(tile_m), int(k_step), int(splits)))


def tgemm_tn(M, N, K, type, A, lda, B, ldb, c_type, C, ldc, alpha=1.0, accumulate=0, workspace=None, workspace_bytes=0,
             stream=None, splits=0, tile_m=0, k_step=0) -> int:
    return int(_ops().tgemm_tn(M, N, K, _code(_DTYPE, type), A, lda, B, ldb, _code(_DTYPE, c_type), C, ldc,
                               float(alpha), int(accumulate), workspace, workspace_bytes, stream, int(tile_m),
                               int(k_step), int(splits)))


def tgemm_tn_workspace(M, N, K, type, lda, ldb, c_type, ldc, splits=0, tile_m=0, k_step=0) -> int:
    return int(_ops().tgemm_tn_workspace(M, N, K, _code(_DTYPE, type), lda, ldb, _code(_DTYPE, c_type), ldc,
                                         int(tile_m), int(k_step), int(splits)))


def tgemm_act_grad(M, N, type, dY, lddy, act, pre, ldpre, dP, lddp, dbias_type="f32", dbias=None, workspace=None,
                   workspace_bytes=0, stream=None) -> int:
    return int(_ops().tgemm_act_grad(M, N, _code(_DTYPE, type), dY, lddy, _code(_ACTS, act), pre, ldpre, dP, lddp,
                                     _code(_DTYPE, dbias_type), dbias, workspace, workspace_bytes, stream))


def tgemm_act_grad_workspace(M, N) -> int:
    return int(_ops().tgemm_act_grad_workspace(M, N))


def tgemm_act_grad_f32(M, N, type, dY, lddy, act, pre, ldpre, dP, lddp, scale, dbias_type="f32", dbias=None,
                       workspace=None, workspace_bytes=0, stream=None) -> int:
    return int(_ops().tgemm_act_grad_f32(M, N, _code(_DTYPE, type), dY, lddy, _code(_ACTS, act), pre, ldpre, dP, lddp, scale,
                                         _code(_DTYPE, dbias_type), dbias, workspace, workspace_bytes, stream))


def tgemm_act_grad_f32_workspace(M, N) -> int:
    return int(_ops().tgemm_act_grad_f32_workspace(M, N))


def tgemm_linear_grad(M, N, K, type, X, ldx, W, ldw, w_layout, act, pre, ldpre, dY, lddy, dX=None, lddx=0, dW=None,
                      lddw=0, dbias_type="f32", dbias=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    return int(_ops().tgemm_linear_grad(M, N, K, _code(_DTYPE, type), X, ldx, W, ldw, _LAYOUT.get(w_layout, w_layout),
                                        _code(_ACTS, act), pre, ldpre, dY, lddy, dX, lddx, dW, lddw,
                                        _code(_DTYPE, dbias_type), dbias, workspace, workspace_bytes, stream))


def tgemm_linear_grad_workspace(M, N, K, type, ldx, ldw, w_layout, act, lddy, lddx, lddw) -> int:
    return int(_ops().tgemm_linear_grad_workspace(M, N, K, _code(_DTYPE, type), ldx, ldw,
                                                  _LAYOUT.get(w_layout, w_layout), _code(_ACTS, act), lddy, lddx, lddw))


def tgemm_linear_grad_f32(M, N, K, type, X, ldx, W, ldw, w_layout, act, pre, ldpre, dY, lddy, dX=None, lddx=0, dW=None,
                          lddw=0, dbias_type="f32", dbias=None, workspace=None, workspace_bytes=0, stream=None) -> int:
    return int(_ops().tgemm_linear_grad_f32(M, N, K, _code(_DTYPE, type), X, ldx, W, ldw, _LAYOUT.get(w_layout, w_layout),
                                            _code(_ACTS, act), pre, ldpre, dY, lddy, dX, lddx, dW, lddw,
                                            _code(_DTYPE, dbias_type), dbias, workspace, workspace_bytes, stream))


def tgemm_linear_grad_f32_workspace(M, N, K, type, ldx, ldw, w_layout, act, lddy, lddx, lddw) -> int:
    return int(_ops().tgemm_linear_grad_f32_workspace(M, N, K, _code(_DTYPE, type), ldx, ldw,
                                                      _LAYOUT.get(w_layout, w_layout), _code(_ACTS, act), lddy, lddx,
                                                      lddw))


def tgemm_xent(rows, vocab, dim, type, H, ldh, W, ldw, target, ignore, reduction, lse, loss, total=None, count=None,
               workspace=None, workspace_bytes=0, stream=None) -> int:
    return int(_ops().tgemm_xent(rows, vocab, dim, _code(_DTYPE, type), H, ldh, W, ldw, target, ignore,
                                 _code(_REDUCE, reduction), lse, loss, total, count, workspace, workspace_bytes, stream))


def tgemm_xent_workspace(rows, vocab, dim, type, ldh, ldw) -> int:
    return int(_ops().tgemm_xent_workspace(rows, vocab, dim, _code(_DTYPE, type), ldh, ldw))


def tgemm_xent_grad(rows, vocab, dim, type, H, ldh, W, ldw, target, ignore, lse, dloss, dloss_stride, count, dlse, dH,
                    lddh, dW, lddw, workspace=None, workspace_bytes=0, stream=None) -> int:
    return int(_ops().tgemm_xent_grad(rows, vocab, dim, _code(_DTYPE, type), H, ldh, W, ldw, target, ignore, lse, dloss,
                                      int(dloss_stride), count, dlse, dH, lddh, dW, lddw, workspace, workspace_bytes,
                                      stream))


def tgemm_xent_grad_workspace(rows, vocab, dim, type, ldh, ldw, lddh, lddw) -> int:
    return int(_ops().tgemm_xent_grad_workspace(rows, vocab, dim, _code(_DTYPE, type), ldh, ldw, lddh, lddw))


def tgemm_xent_both(rows, vocab, dim, type, H, ldh, W, ldw, target, ignore, reduction, lse, loss, total, count, dH, lddh,
                    dW, lddw, workspace=None, workspace_bytes=0, stream=None) -> int:
    return int(_ops().tgemm_xent_both(rows, vocab, dim, _code(_DTYPE, type), H, ldh, W, ldw, target, ignore,
                                      _code(_REDUCE, reduction), lse, loss, total, count, dH, lddh, dW, lddw, workspace,
                                      workspace_bytes, stream))


def tgemm_xent_both_workspace(rows, vocab, dim, type, ldh, ldw, lddh, lddw) -> int:
    return int(_ops().tgemm_xent_both_workspace(rows, vocab, dim, _code(_DTYPE, type), ldh, ldw, lddh, lddw))


def tgemm_scale(type, n, X, n2, X2, factor, stream=None) -> int:
    return int(_ops().tgemm_scale(_code(_DTYPE, type), n, X, n2, X2, factor, stream))


# ----------------------------------------------------------- torch tensors --

# Workspace sizes depend on sizes, strides and the device alone.
@lru_cache(maxsize=4096)
def _ws_size(device, fn, *args):
    n = int(getattr(_ops(), fn)(*args))
    if n < 0:
        raise TgemmError(n, f"{fn}{args}")
    return n


def _alloc(torch, nbytes, device):
    """(tensor or None, pointer or None) of a workspace on the current stream."""
    if nbytes == 0:
        return None, None
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


_CODES = {}


def _type16(torch, t, name):
    if not _CODES:
        _CODES[torch.bfloat16], _CODES[torch.float16] = TGEMM_BF16, TGEMM_F16
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return code


def _device(t, name, like=None):
    if like is not None:
        if t.device != like:
            raise ValueError(f"{name} is on {t.device}, the first operand on {like}")
    elif not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def _no_tangents(torch, *operands):
    """The functions have no forward-mode derivative: an operand that carries a
    tangent is refused (a call without gradients would drop it)."""
    fw = torch.autograd.forward_ad
    if fw._current_level >= 0 and any(t is not None and fw.unpack_dual(t).tangent is not None for t in operands):
        raise NotImplementedError("no forward-mode derivative: an operand carries a tangent")


def _rows(t):
    """Row stride of a 2-D tensor that the kernels can read as it lies, or None:
    unit column stride and rows that do not overlap."""
    r, c = t.shape
    s, one = t.stride()
    if one != 1 and c > 1:
        return None
    if r <= 1:
        return c or 1
    return s if s >= c and s >= 1 else None


def _readable(t):
    """t itself where the kernels can read it, otherwise a contiguous copy
    (transposed, broadcast or overlapping rows)."""
    ld = _rows(t)
    if ld is None:
        t = t.contiguous()
        ld = max(t.shape[1], 1)
    return t, ld


# Rows of the cross entropy's operands and of a residual lie at most this many elements apart.
_MAX_LD = 4000000


def _near(t):
    """t, or a contiguous copy where its rows lie further apart than _MAX_LD."""
    return t.contiguous() if (_rows(t) or 0) > _MAX_LD else t


class _Here:
    """The device is the current one already."""
    def __enter__(self):
        pass

    def __exit__(self, *e):
        pass


_HERE = _Here()


def _On(torch, device):
    """The operands' device as the current one."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stream(torch, device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _linear(torch, x, w, bias, act, residual, out_dtype, layout, keep_pre, tile_m=0, splits=0, k_step=0):
    """(y, pre or None) of 2-D operands whose arguments have been checked."""
    M, K = x.shape
    N = w.shape[0] if layout == TGEMM_B_NxK else w.shape[1]
    dev = x.device
    code = _type16(torch, x, "x")
    x, ldx = _readable(x)
    w, ldw = _readable(w)
    with _On(torch, dev):
        y = x.new_empty((M, N), dtype=out_dtype)
        pre = x.new_empty((M, N)) if keep_pre else None
        y_code = TGEMM_F32 if out_dtype == torch.float32 else code
        ldy = max(N, 1)
        need = _ws_size(dev.index, "tgemm_linear_config_workspace", M, N, K, code, ldx, ldw, layout, y_code, ldy,
                        tile_m, k_step, splits)
        ldr = 0
        if residual is not None:
            residual, ldr = _readable(residual)
            if ldr > _MAX_LD >= N:
                residual, ldr = residual.contiguous(), ldy
        ws, ws_ptr = _alloc(torch, need, dev)
        b_code = TGEMM_F32
        if bias is not None:
            if N > 1 and bias.stride(0) != 1:
                bias = bias.contiguous()
            if bias.dtype != torch.float32:
                b_code = code
        rc = _ops().tgemm_linear_config(
            M, N, K, code, x.data_ptr(), ldx, w.data_ptr(), ldw, layout, None if bias is None else bias.data_ptr(),
            b_code, _ACTS[act], None if residual is None else residual.data_ptr(), ldr, y_code, y.data_ptr(), ldy,
            None if pre is None else pre.data_ptr(), ldy, 1.0, ws_ptr, need, _stream(torch, dev), tile_m,
            k_step, splits)
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"linear M={M} N={N} K={K} {x.dtype}->{out_dtype} act={act}")
    return y, pre


def _linear_grad(torch, x, w, act, pre, dy, layout, need_x, need_w, bias_dtype):
    """(dx, dw, db) of 2-D operands as the forward call took them; dy of the
    operands' dtype or (an fp32 result's) float32."""
    M, K = x.shape
    N = dy.shape[1]
    dev = x.device
    dt = x.dtype
    code = TGEMM_BF16 if dt == torch.bfloat16 else TGEMM_F16
    fn = "tgemm_linear_grad" if dy.dtype == dt else "tgemm_linear_grad_f32"
    x, ldx = _readable(x)
    w, ldw = _readable(w)
    dy, lddy = _readable(dy)
    act = _ACTS[act]
    ldn, ldk = N or 1, K or 1
    lddw = ldk if layout == TGEMM_B_NxK else ldn
    with _On(torch, dev):
        dx = torch.empty((M, K), dtype=dt, device=dev) if need_x else None
        dw = torch.empty(w.shape, dtype=dt, device=dev) if need_w else None
        db = None if bias_dtype is None else torch.empty((N,), dtype=bias_dtype, device=dev)
        need = _ws_size(dev.index, fn + "_workspace", M, N, K, code, ldx, ldw, layout, act, lddy, ldk, lddw)
        ws, ws_ptr = _alloc(torch, need, dev)
        rc = getattr(_ops(), fn)(
            M, N, K, code, x.data_ptr(), ldx, w.data_ptr(), ldw, layout, act, None if pre is None else pre.data_ptr(), ldn,
            dy.data_ptr(), lddy, None if dx is None else dx.data_ptr(), ldk, None if dw is None else dw.data_ptr(), lddw,
            TGEMM_F32 if bias_dtype == torch.float32 else code, None if db is None else db.data_ptr(), ws_ptr, need,
            _stream(torch, dev))
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"linear backward M={M} N={N} K={K} {dt} act={act}")
    return dx, dw, db


def gemm_tn(A, B, out=None, out_dtype=None, alpha: float = 1.0, accumulate: bool = False, splits: int = 0,
            tile_m: int = 0, k_step: int = 0):
    """C = alpha * A^T @ B (+ out where ``accumulate``) for float16 or bfloat16
    device tensors A (K, M) and B (K, N), fp32 accumulation: a weight gradient
    from activations and gradients as they lie.

    out: optional (M, N) tensor with unit column stride, of A's dtype or
    float32; allocated as ``out_dtype`` (default A's dtype) when None. splits,
    tile_m, k_step: explicit launch choices (tgemm_tn). A part of gradients: it
    takes no part in autograd itself, its result has no history.
    """
    import torch
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    _device(A, "A")
    _device(B, "B", A.device)
    code = _type16(torch, A, "A")
    if B.dtype != A.dtype:
        raise TypeError(f"A and B must be of one dtype, got {A.dtype} and {B.dtype}")
    K, M = A.shape
    N = B.shape[1]
    if B.shape[0] != K:
        raise ValueError(f"the long axes differ: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    _no_tangents(torch, A, B, out)
    given = out is not None
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        with _On(torch, A.device):
            out = torch.empty((M, N), dtype=out_dtype or A.dtype, device=A.device)
    elif tuple(out.shape) != (M, N):
        raise ValueError(f"out must be ({M}, {N})")
    elif out_dtype is not None and out_dtype != out.dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    _device(out, "out", A.device)
    if out.dtype not in (A.dtype, torch.float32):
        raise TypeError(f"out must be {A.dtype} or float32, got {out.dtype}")
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out requires a gradient; writes have no history")
    ldc = _rows(out)
    if ldc is None:
        raise ValueError("out must have unit column stride and rows that do not overlap")
    A, lda = _readable(A)
    B, ldb = _readable(B)
    c_code = TGEMM_F32 if out.dtype == torch.float32 else code
    dev = A.device
    with _On(torch, dev):
        need = _ws_size(dev.index, "tgemm_tn_workspace", M, N, K, code, lda, ldb, c_code, ldc, tile_m, k_step,
                        splits)
        ws, ws_ptr = _alloc(torch, need, dev)
        rc = _ops().tgemm_tn(M, N, K, code, A.data_ptr(), lda, B.data_ptr(), ldb, c_code, out.data_ptr(), ldc,
                             alpha, 1 if accumulate else 0, ws_ptr, need, _stream(torch, dev), tile_m, k_step, splits)
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"gemm_tn M={M} N={N} K={K} {A.dtype}->{out.dtype}")
    if given and not out.is_inference():
        torch.autograd.graph.increment_version(out)   # what autograd has saved of out is stale
    return out


def act_grad(dy, act: str, pre=None, bias_dtype=None):
    """(dp, db): dp = dy * act'(pre) of dy's dtype (dy itself for "none"), and
    its column sums, taken before dp is rounded, as ``bias_dtype`` (dy's dtype
    or float32; None: not computed). dy, pre: (M, N) float16 or bfloat16. A part
    of gradients: the results have no history in autograd."""
    import torch
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    if dy.dim() != 2:
        raise ValueError("dy must be 2-D")
    _device(dy, "dy")
    code = _type16(torch, dy, "dy")
    M, N = dy.shape
    dev = dy.device
    if bias_dtype not in (None, dy.dtype, torch.float32):
        raise TypeError(f"bias_dtype must be {dy.dtype} or float32, got {bias_dtype}")
    _no_tangents(torch, dy)
    dy, lddy = _readable(dy)
    pre_ptr = dp_ptr = None
    ldpre = lddp = 0
    dp = dy
    with _On(torch, dev):
        if act != "none":
            if pre is None or tuple(pre.shape) != (M, N) or pre.dtype != dy.dtype:
                raise ValueError(f"pre must be a ({M}, {N}) {dy.dtype} tensor")
            _device(pre, "pre", dev)
            _no_tangents(torch, pre)
            pre, ldpre = _readable(pre)
            dp = torch.empty((M, N), dtype=dy.dtype, device=dev)
            lddp = max(N, 1)
            pre_ptr, dp_ptr = pre.data_ptr(), dp.data_ptr()
        db, need = None, 0
        if bias_dtype is not None:
            db = torch.empty((N,), dtype=bias_dtype, device=dev)
            need = _ws_size(dev.index, "tgemm_act_grad_workspace", M, N)
        elif act == "none":
            return dy, None
        ws, ws_ptr = _alloc(torch, need, dev)
        rc = _ops().tgemm_act_grad(M, N, code, dy.data_ptr(), lddy, _ACTS[act], pre_ptr, ldpre, dp_ptr, lddp,
                                   TGEMM_F32 if bias_dtype == torch.float32 else code,
                                   None if db is None else db.data_ptr(), ws_ptr, need, _stream(torch, dev))
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"act_grad M={M} N={N} {dy.dtype} act={act}")
    return dp, db


_fns = {}


def _functions():
    """The autograd functions (built on first use: torch is imported lazily)."""
    if _fns:
        return _fns
    import torch

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, bias, residual, act, out_dtype, layout):
            keep = act != "none" and any(ctx.needs_input_grad[:3])
            y, pre = _linear(torch, x, w, bias, act, residual, out_dtype, layout, keep)
            ctx.save_for_backward(x, w, pre)
            ctx.act, ctx.layout = act, layout
            ctx.bias_dtype = None if bias is None else bias.dtype
            ctx.res_dtype = None if residual is None else residual.dtype
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, w, pre = ctx.saved_tensors
            nx, nw, nb, nr = ctx.needs_input_grad[:4]
            dx = dw = db = dres = None
            if nr:
                dres = dy if dy.dtype == ctx.res_dtype else dy.to(ctx.res_dtype)
            if nx or nw or nb:
                dx, dw, db = _linear_grad(torch, x, w, ctx.act, pre, dy, ctx.layout, nx, nw, ctx.bias_dtype if nb else None)
            return dx, dw, db, dres, None, None, None

    class CrossEntropy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, w, target, ignore, reduction, both):
            ctx.set_materialize_grads(False)
            ctx.ignore, ctx.reduction = ignore, reduction
            ctx.grads = None
            if both:
                loss, lse, total, count, *ctx.grads = _xent_both(torch, h, w, target, ignore, reduction,
                                                                 *ctx.needs_input_grad[:2])
            else:
                loss, lse, total, count = _xent(torch, h, w, target, ignore, reduction)
            ctx.save_for_backward(h, w, target, lse, count)
            return (loss if total is None else total), lse

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dloss, dlse):
            h, w, target, lse, count = ctx.saved_tensors
            grads, ctx.grads = ctx.grads, None
            if grads is not None and dlse is None and dloss is not None:
                # the forward pass's gradients, handed out once; a second pass recomputes
                _scale(torch, *grads, dloss)
                return (*grads, None, None, None, None)
            dh, dw = _xent_grad(torch, h, w, target, lse, dloss, dlse, count if ctx.reduction == "mean" else None,
                                ctx.ignore, ctx.needs_input_grad[0], ctx.needs_input_grad[1])
            return dh, dw, None, None, None, None

    _fns["linear"], _fns["xent"] = Linear, CrossEntropy
    return _fns


def linear(x, weight, bias=None, act: str = "none", residual=None, out_dtype=None, w_layout: str = "NxK",
           tile_m: int = 0, splits: int = 0, k_step: int = 0):
    """act(x @ weight^T + bias) + residual for float16 or bfloat16 device
    tensors, fp32 accumulation and epilogue, one rounding of the result.

    x: (..., K). weight: (N, K), or (K, N) with ``w_layout="KxN"``. bias: None or
    (N,) of x's dtype or float32. act: "none", "relu", "silu", "gelu" (erf) or
    "gelu_tanh". residual: None or (..., N) of x's dtype. out_dtype: x's dtype
    (default) or float32. Operands may have any row stride; what is not
    row-major is copied first.

    Differentiable in x, weight, bias and residual. With an activation the
    backward pass keeps the pre-activation in x's dtype. The result's gradient,
    times the activation's derivative, is rounded once to x's dtype for the
    products (bias gradients sum it unrounded); where the result is float32 and x
    float16 it is scaled by its largest value for that, so that gradients below
    2^-25 and above 65504 keep their precision. tile_m, splits, k_step: explicit
    launch choices (tgemm_linear_config), without autograd.
    """
    import torch
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    if w_layout not in ("NxK", "KxN"):
        raise ValueError(f"w_layout must be 'NxK' or 'KxN', got {w_layout!r}")
    layout = _LAYOUT[w_layout]
    _device(x, "x")
    dev = x.device
    dt = x.dtype
    _type16(torch, x, "x")
    if weight.dim() != 2 or x.dim() < 1:
        raise ValueError("weight must be 2-D and x at least 1-D")
    if weight.dtype != dt:
        raise TypeError(f"x and weight must be of one dtype, got {dt} and {weight.dtype}")
    _device(weight, "weight", dev)
    N, K = weight.shape if layout == TGEMM_B_NxK else (weight.shape[1], weight.shape[0])
    if x.shape[-1] != K:
        raise ValueError(f"inner dimensions differ: x is {tuple(x.shape)}, weight {tuple(weight.shape)} ({w_layout})")
    if out_dtype is None:
        out_dtype = dt
    elif out_dtype not in (dt, torch.float32):
        raise TypeError(f"out_dtype must be {dt} or float32, got {out_dtype}")
    if bias is not None:
        if bias.shape != (N,) or bias.dtype not in (dt, torch.float32):
            raise ValueError(f"bias must be a ({N},) tensor of {dt} or float32")
        _device(bias, "bias", dev)
    shape = x.shape[:-1] + (N,)
    if residual is not None:
        if residual.shape != shape or residual.dtype != dt:
            raise ValueError(f"residual must be a {tuple(shape)} tensor of {dt}")
        _device(residual, "residual", dev)
    _no_tangents(torch, x, weight, bias, residual)
    if x.dim() != 2:
        rows = 1
        for s in x.shape[:-1]:
            rows *= s
        x = x.reshape(rows, K)
        if residual is not None:
            residual = residual.reshape(rows, N)
    grad = torch.is_grad_enabled() and (
        x.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad)
        or (residual is not None and residual.requires_grad))
    if grad:
        if tile_m or splits or k_step:
            raise ValueError("tile_m, splits and k_step are for calls without gradients")
        y = _functions()["linear"].apply(x, weight, bias, residual, act, out_dtype, layout)
    else:
        y, _ = _linear(torch, x, weight, bias, act, residual, out_dtype, layout, False, tile_m, splits, k_step)
    return y if len(shape) == 2 else y.reshape(shape)


def _xent(torch, h, w, target, ignore, reduction):
    """(losses, lse, total or None, count or None)."""
    R, D = h.shape
    V = w.shape[0]
    dev = h.device
    code = _type16(torch, h, "hidden")
    h, ldh = _readable(h)
    w, ldw = _readable(w)
    target = target.contiguous()
    with _On(torch, dev):
        loss = torch.empty((R,), dtype=torch.float32, device=dev)
        lse = torch.empty((R,), dtype=torch.float32, device=dev)
        total = count = None
        if reduction != "none":
            total = torch.empty((), dtype=torch.float32, device=dev)
            count = torch.empty((), dtype=torch.float32, device=dev)
        need = _ws_size(dev.index, "tgemm_xent_workspace", R, V, D, code, ldh, ldw)
        ws, ws_ptr = _alloc(torch, need, dev)
        rc = _ops().tgemm_xent(R, V, D, code, h.data_ptr(), ldh, w.data_ptr(), ldw, target.data_ptr(), ignore,
                               _REDUCE[reduction], lse.data_ptr(), loss.data_ptr(),
                               None if total is None else total.data_ptr(),
                               None if count is None else count.data_ptr(), ws_ptr, need, _stream(torch, dev))
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"linear_cross_entropy rows={R} vocab={V} dim={D} {h.dtype}")
    return loss, lse, total, count


# Rows from which the loss and its gradients are computed together.
_BOTH_ROWS = 33


@lru_cache(maxsize=4096)
def _both_fits(device, R, V, D, code, ldh, ldw):
    """Whether tgemm_xent_both takes these sizes (its type and workspace rules)."""
    import torch
    with _On(torch, torch.device("cuda", device)):
        return int(_ops().tgemm_xent_both_workspace(R, V, D, code, ldh, ldw, D, D)) >= 0


def _both_ok(torch, h, w):
    R, D = h.shape
    return R >= _BOTH_ROWS and _both_fits(h.device.index, R, w.shape[0], D, _type16(torch, h, "hidden"), _rows(h) or D,
                                          _rows(w) or D)


def _xent_both(torch, h, w, target, ignore, reduction, need_h, need_w):
    """(losses, lse, total, count, dh, dw) for a loss gradient of 1."""
    R, D = h.shape
    V = w.shape[0]
    dev = h.device
    code = _type16(torch, h, "hidden")
    h2, ldh = _readable(h)
    w2, ldw = _readable(w)
    target = target.contiguous()
    with _On(torch, dev):
        loss = torch.empty((R,), dtype=torch.float32, device=dev)
        lse = torch.empty((R,), dtype=torch.float32, device=dev)
        total = torch.empty((), dtype=torch.float32, device=dev)
        count = torch.empty((), dtype=torch.float32, device=dev)
        dh = torch.empty((R, D), dtype=h.dtype, device=dev) if need_h else None
        dw = torch.empty((V, D), dtype=w.dtype, device=dev) if need_w else None
        need = _ws_size(dev.index, "tgemm_xent_both_workspace", R, V, D, code, ldh, ldw, D, D)
        ws, ws_ptr = _alloc(torch, need, dev)
        rc = _ops().tgemm_xent_both(R, V, D, code, h2.data_ptr(), ldh, w2.data_ptr(), ldw, target.data_ptr(), ignore,
                                    _REDUCE[reduction], lse.data_ptr(), loss.data_ptr(), total.data_ptr(),
                                    count.data_ptr(), None if dh is None else dh.data_ptr(), D,
                                    None if dw is None else dw.data_ptr(), D, ws_ptr, need, _stream(torch, dev))
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"linear_cross_entropy with gradients rows={R} vocab={V} dim={D} {h.dtype}")
    return loss, lse, total, count, dh, dw


def _scale(torch, a, b, factor):
    """a and b (each a tensor or None) *= factor (one value) in place."""
    factor = factor.float()
    a, b = (b, None) if a is None else (a, b)
    if a is None:
        return
    with _On(torch, a.device):
        rc = _ops().tgemm_scale(_type16(torch, a, "gradient"), a.numel(), a.data_ptr(), 0 if b is None else b.numel(),
                                None if b is None else b.data_ptr(), factor.data_ptr(), _stream(torch, a.device))
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"scale of {a.numel()} {a.dtype}")


def _xent_grad(torch, h, w, target, lse, dloss, dlse, count, ignore, need_h, need_w):
    R, D = h.shape
    V = w.shape[0]
    dev = h.device
    code = _type16(torch, h, "hidden")
    h2, ldh = _readable(h)
    w2, ldw = _readable(w)
    target = target.contiguous()
    stride = 0
    if dloss is not None:
        dloss = dloss.float()
        if dloss.dim() == 1:
            stride = 1
            dloss = dloss.contiguous()
    if dlse is not None:
        dlse = dlse.float().contiguous()
    with _On(torch, dev):
        dh = torch.empty((R, D), dtype=h.dtype, device=dev) if need_h else None
        dw = torch.empty((V, D), dtype=w.dtype, device=dev) if need_w else None
        need = _ws_size(dev.index, "tgemm_xent_grad_workspace", R, V, D, code, ldh, ldw, D, D)
        ws, ws_ptr = _alloc(torch, need, dev)
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        rc = _ops().tgemm_xent_grad(R, V, D, code, h2.data_ptr(), ldh, w2.data_ptr(), ldw, target.data_ptr(), ignore,
                                    lse.data_ptr(), ptr(dloss), stride, ptr(count), ptr(dlse), ptr(dh), D, ptr(dw), D,
                                    ws_ptr, need, _stream(torch, dev))
    if rc != TGEMM_OK:
        raise TgemmError(rc, f"linear_cross_entropy backward rows={R} vocab={V} dim={D} {h.dtype}")
    return dh, dw


def linear_cross_entropy(hidden, weight, target, ignore_index: int = -100, reduction: str = "mean",
                         return_lse: bool = False, recompute: bool = False):
    """Softmax cross entropy of the logits ``hidden @ weight^T`` against
    ``target``, without keeping the logits.

    hidden: (..., D) and weight: (V, D), float16 or bfloat16 device tensors, D >=
    8; target: (...) int64. Rows whose target is ``ignore_index`` have loss 0 and
    pass no gradient. reduction: "none" (float32 losses of target's shape),
    "sum" or "mean" (over the rows that are not ignored; 0 where there is none).
    return_lse: also the rows' log-sum-exp, float32 of target's shape
    (differentiable: a penalty on it needs no second pass).

    A target outside the vocabulary (and not ``ignore_index``) gives NaN.
    Differentiable in hidden and weight. An ignored row's hidden state has to be
    finite. For a "sum" or "mean" of bfloat16 operands without return_lse, of 33
    rows or more, a call under autograd computes the gradients at once, from
    16-bit exponentials that live for the call (2 bytes a logit, as much as
    16-bit logits take), where rows times the vocabulary rounded up to an odd
    multiple of 64 is at most 2^30. It keeps the gradients (of the operands'
    sizes) for the backward pass, which multiplies them by the loss's gradient
    (one more rounding where that is no power of two) and does nothing where it
    is 1; they are no saved tensors, so hooks on those do not see them, and a
    checkpointed call computes them twice. Elsewhere, in a second backward pass,
    and with ``recompute=True`` (a loss that may see no backward pass, a
    checkpoint, memory that has no room for the logits), the forward pass keeps
    the rows' log-sum-exp alone and the backward pass computes the logits again
    in pieces of the vocabulary of at most 2^28 of them.
    """
    import torch
    if reduction not in _REDUCE:
        raise ValueError(f"reduction must be 'none', 'sum' or 'mean', got {reduction!r}")
    _device(hidden, "hidden")
    dev = hidden.device
    _type16(torch, hidden, "hidden")
    if weight.dim() != 2 or hidden.dim() < 1:
        raise ValueError("weight must be 2-D and hidden at least 1-D")
    if weight.dtype != hidden.dtype:
        raise TypeError(f"hidden and weight must be of one dtype, got {hidden.dtype} and {weight.dtype}")
    _device(weight, "weight", dev)
    V, D = weight.shape
    if hidden.shape[-1] != D:
        raise ValueError(f"inner dimensions differ: hidden is {tuple(hidden.shape)}, weight {tuple(weight.shape)}")
    if D < 8 or V < 1:
        raise ValueError(f"weight must have at least one row of at least 8 values, got {tuple(weight.shape)}")
    shape = hidden.shape[:-1]
    if target.dtype != torch.int64 or target.shape != shape:
        raise ValueError(f"target must be a {tuple(shape)} int64 tensor")
    _device(target, "target", dev)
    _no_tangents(torch, hidden, weight)
    rows = target.numel()
    if rows == 0 and reduction != "none":
        # the sum over no rows (a mean divides by one at least)
        loss, lse = linear_cross_entropy(hidden, weight, target, ignore_index, "none", True)
        return (loss.sum(), lse) if return_lse else loss.sum()
    h = _near(hidden if hidden.dim() == 2 else hidden.reshape(rows, D))
    weight = _near(weight)
    t = target.reshape(rows)
    if torch.is_grad_enabled() and (h.requires_grad or weight.requires_grad):
        both = not recompute and not return_lse and reduction != "none" and _both_ok(torch, h, weight)
        out, lse = _functions()["xent"].apply(h, weight, t, int(ignore_index), reduction, both)
    else:
        loss, lse, total, _ = _xent(torch, h, weight, t, int(ignore_index), reduction)
        out = loss if total is None else total
    if reduction == "none":
        out = out.reshape(shape)
    return (out, lse.reshape(shape)) if return_lse else out
