"""ctypes binding of libmoe_block: the same names as include/moe_block.h.

Every function takes torch tensors that already live on one GPU, checks what
the C ABI cannot see (types, shapes, devices, that a row's elements are
adjacent), passes raw pointers and strides on the current stream of that GPU
(or ``stream``) and raises ``MoEError`` on a non-OK status.  Matrices are
two-dimensional [rows, H], fp32 or bf16, and may be strided by rows; vectors
and the [T, k] arrays are contiguous.  No arithmetic happens in Python, and
there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import re
import threading

import torch

from . import _lib
from . import build as _build
from ._lib import MOE_EINVAL, MOE_ENOTSUP, MOE_ESHAPE, MOE_OK, MoEError

MOE_ROW_F32, MOE_ROW_BF16 = 0, 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = range(4)

HEADER = os.path.join(_build.INCLUDE, "moe_block.h")

_lock = threading.Lock()
_blk = None

_TYPES = {torch.float32: MOE_ROW_F32, torch.bfloat16: MOE_ROW_BF16}


def declared_functions():
    """Names of the functions include/moe_block.h declares (parsed from the header)."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"MOE_API\s+[\w\s\*]*?\b(moe_\w+)\s*\(", txt)))


def load():
    """Load (building first if needed) libmoe_block.so and declare its signatures."""
    global _blk
    if _blk is not None:
        return _blk
    with _lock:
        if _blk is not None:
            return _blk
        lib = C.CDLL(_build.build(lib=_build.LIB_BLOCK))
        p, i, l, f, sz = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t
        sig = {
            "moe_block_abi_version": ([], i),
            "moe_dispatch": ([p, l, i, p, p, i, i, i, i, p, l, p, p], i),
            "moe_dispatch_backward": ([p, l, i, p, p, p, l, i, i, i, i, p, l, i, p, l, p, p, p], i),
            "moe_collect": ([p, l, i, p, p, i, i, i, i, p, l, i, p, l, p, p], i),
            "moe_collect_backward": ([p, l, i, p, l, i, p, p, i, i, i, i, p, l, p, p, p], i),
            "moe_block_norm": ([p, l, i, p, l, i, p, i, l, p, p, i, f, f, i, i, p, l, p, l, p, p, p], i),
            "moe_block_norm_workspace_size": ([i, i], sz),
            "moe_block_norm_backward": ([p, l, p, l, p, l, i, p, l, i, p, i, l, p, p, i, f, p, p, i, i, p, l, p, l, p, l,
                                         p, p, p, sz, p], i),
            "moe_route_backward_workspace_size": ([i, i, i, i], sz),
            "moe_route_backward": ([p, p, p, p, l, p, l, p, p, i, i, i, i, p, p, l, i, p, l, p, l, p, p, sz, p, p], i),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _blk = lib
        return lib


# The checks of a call.  ``fn`` is its name, ``dev`` the GPU of its tensors (-1:
# they are on the CPU).
def _no(fn, status, what):
    raise MoEError(fn, status, what)


def _matrix(fn, t, name):
    """(rows, width, type, GPU) of the matrix that the others are measured by."""
    if t.dim() != 2:
        _no(fn, MOE_ESHAPE, f"{name} must be two-dimensional")
    n, H = t.shape
    return n, H, _type(fn, t, name), t.get_device()


def _type(fn, t, name):
    ty = _TYPES.get(t.dtype)
    if ty is None:
        _no(fn, MOE_EINVAL, f"{name} has type {t.dtype}, expected float32 or bfloat16")
    return ty


def _tensor_no(fn, dev, t, name, shape, dtype):
    if t.get_device() != dev or dev < 0:
        _no(fn, MOE_EINVAL, f"{name} is not on GPU {dev}" if dev >= 0 else "tensors must be on a GPU")
    if t.shape != shape:
        _no(fn, MOE_ESHAPE, f"{name} has shape {tuple(t.shape)}, expected {shape}")
    _no(fn, MOE_EINVAL, f"{name} has type {t.dtype}, expected {dtype}")


def _rows(fn, dev, t, name, n, H, dtype):
    """(pointer, row stride) of a [n, H] matrix; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.get_device() != dev or t.dtype is not dtype or t.shape != (n, H) or dev < 0:
        _tensor_no(fn, dev, t, name, (n, H), dtype)
    if n > 0x7fffffff or H > 0x7fffffff:
        _no(fn, MOE_ENOTSUP, f"{name} has shape {(n, H)}: sizes are 32-bit")
    ld, step = t.stride()
    if step != 1 and H > 1:
        _no(fn, MOE_EINVAL, f"{name}: the elements of a row must be adjacent")
    return t.data_ptr(), ld if n > 1 else max(ld, H)


def _flat(fn, dev, t, name, shape, dtype=torch.float32):
    """Pointer of a contiguous array; None for None."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or dev < 0:
        _tensor_no(fn, dev, t, name, shape, dtype)
    if not t.is_contiguous():
        _no(fn, MOE_EINVAL, f"{name} is not contiguous")
    return t.data_ptr()


def _bytes(fn, dev, t, name):
    """(pointer, size in bytes) of a workspace; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.get_device() != dev or dev < 0:
        _no(fn, MOE_EINVAL, f"{name} is not on GPU {dev}")
    if not t.is_contiguous():
        _no(fn, MOE_EINVAL, f"{name} is not contiguous")
    return t.data_ptr(), t.nbytes


def _routes(fn, dev, inv_perm, T, name="inv_perm"):
    if inv_perm.dim() != 2:
        _no(fn, MOE_ESHAPE, f"{name} must be [T, k]")
    k = inv_perm.shape[1]
    return k, _flat(fn, dev, inv_perm, name, (T, k), torch.int32)


_functions = {}


def _issue(fn, dev, stream, args):
    """The C call with the GPU of its tensors current, on `stream` or that GPU's current stream."""
    f = _functions.get(fn)
    if f is None:
        f = _functions[fn] = getattr(load(), fn)
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != MOE_OK:
        raise MoEError(fn, st, _lib.status_str(st))


def moe_dispatch(x, inv_perm, x_perm, w=None, dev_status=None, stream=None):
    """x_perm[inv_perm[t,j]] = w[t,j] * x[t] (w None: 1); routes of slot -1 and rows without a route are left out."""
    fn = "moe_dispatch"
    T, H, ty, dev = _matrix(fn, x, "x")
    k, inv = _routes(fn, dev, inv_perm, T)
    R = len(x_perm)
    px, ldx = _rows(fn, dev, x, "x", T, H, x.dtype)
    pp, ldp = _rows(fn, dev, x_perm, "x_perm", R, H, x.dtype)
    _issue(fn, dev, stream, (px, ldx, ty, inv, _flat(fn, dev, w, "w", (T, k)), T, k, H, R, pp, ldp,
                             _flat(fn, dev, dev_status, "dev_status", (1,), torch.int32)))


def moe_dispatch_backward(dx_perm, inv_perm, dx, w=None, x=None, dw=None, add=None, dev_status=None, stream=None):
    """dx = add + sum_j w * dx_perm[inv_perm]; with dw (and x), dw[t,j] = <dx_perm[inv_perm[t,j]], x[t]>."""
    fn = "moe_dispatch_backward"
    T, H, dty, dev = _matrix(fn, dx, "dx")
    k, inv = _routes(fn, dev, inv_perm, T)
    R, ty = len(dx_perm), _type(fn, dx_perm, "dx_perm")
    pp, ldp = _rows(fn, dev, dx_perm, "dx_perm", R, H, dx_perm.dtype)
    px, ldx = _rows(fn, dev, x, "x", T, H, dx_perm.dtype)
    pd, ldd = _rows(fn, dev, dx, "dx", T, H, dx.dtype)
    pa, lda = _rows(fn, dev, add, "add", T, H, dx.dtype)
    _issue(fn, dev, stream, (pp, ldp, ty, inv, _flat(fn, dev, w, "w", (T, k)), px, ldx, T, k, H, R, pd, ldd, dty, pa, lda,
                             _flat(fn, dev, dw, "dw", (T, k)),
                             _flat(fn, dev, dev_status, "dev_status", (1,), torch.int32)))


def moe_collect(y_perm, inv_perm, w, out, add=None, dev_status=None, stream=None):
    """out = add + sum_j w * y_perm[inv_perm] in rank order (w None: 1)."""
    fn = "moe_collect"
    T, H, oty, dev = _matrix(fn, out, "out")
    k, inv = _routes(fn, dev, inv_perm, T)
    R, ty = len(y_perm), _type(fn, y_perm, "y_perm")
    pp, ldp = _rows(fn, dev, y_perm, "y_perm", R, H, y_perm.dtype)
    po, ldo = _rows(fn, dev, out, "out", T, H, out.dtype)
    pa, lda = _rows(fn, dev, add, "add", T, H, out.dtype)
    _issue(fn, dev, stream, (pp, ldp, ty, inv, _flat(fn, dev, w, "w", (T, k)), T, k, H, R, po, ldo, oty, pa, lda,
                             _flat(fn, dev, dev_status, "dev_status", (1,), torch.int32)))


def moe_collect_backward(dout, y_perm, inv_perm, w, dy_perm, dw=None, dev_status=None, stream=None):
    """dy_perm[inv_perm[t,j]] = w[t,j] * dout[t]; with dw (and y_perm), dw[t,j] = <dout[t], y_perm[inv_perm[t,j]]>."""
    fn = "moe_collect_backward"
    T, H, oty, dev = _matrix(fn, dout, "dout")
    k, inv = _routes(fn, dev, inv_perm, T)
    R, ty = len(dy_perm), _type(fn, dy_perm, "dy_perm")
    po, ldo = _rows(fn, dev, dout, "dout", T, H, dout.dtype)
    py, ldy = _rows(fn, dev, y_perm, "y_perm", R, H, dy_perm.dtype)
    pd, ldd = _rows(fn, dev, dy_perm, "dy_perm", R, H, dy_perm.dtype)
    _issue(fn, dev, stream, (po, ldo, oty, py, ldy, ty, inv, _flat(fn, dev, w, "w", (T, k)), T, k, H, R, pd, ldd,
                             _flat(fn, dev, dw, "dw", (T, k)),
                             _flat(fn, dev, dev_status, "dev_status", (1,), torch.int32)))


def _gate(fn, dev, gate, name, T, H, dtype, kind=None):
    """(kind, pointer, row stride): [H] per channel, [T, 1] per token, [T, H] elementwise (of y's type)."""
    if gate is None:
        return MOE_GATE_NONE, None, 0
    if kind is None:
        if gate.dim() == 1:
            kind = MOE_GATE_CHANNEL
        elif gate.shape[1:] == (1,) and gate.dtype is torch.float32 and (H > 1 or dtype is not torch.float32):
            kind = MOE_GATE_TOKEN
        else:
            kind = MOE_GATE_FULL
    if kind == MOE_GATE_CHANNEL:
        return kind, _flat(fn, dev, gate, name, (H,)), 0
    if kind == MOE_GATE_TOKEN:
        return kind, _flat(fn, dev, gate, name, (T, 1)), 0
    return (kind,) + _rows(fn, dev, gate, name, T, H, dtype)


def moe_block_norm(x, y, x_out, n_out, gamma_post=None, gamma_pre=None, gate=None, scale=1.0, eps=1e-6,
                   post_norm=True, rstd_post=None, rstd_pre=None, stream=None):
    """x_out = scale * x + gate * RMSNorm(y), n_out = RMSNorm(x_out), in one pass.

    y None: no block before it (x_out = scale * x); x_out or n_out None: not
    wanted.  gate: [H], [T, 1] (both fp32) or [T, H] of y's type.  The norms'
    gain is 1 + gamma; post_norm=False leaves y as it is.
    """
    fn = "moe_block_norm"
    T, H, xty, dev = _matrix(fn, x, "x")
    act = y if y is not None else n_out
    if act is None:
        _no(fn, MOE_EINVAL, "y and n_out are both None")
    yty, yt = _type(fn, act, "y" if y is not None else "n_out"), act.dtype
    px, ldx = _rows(fn, dev, x, "x", T, H, x.dtype)
    py, ldy = _rows(fn, dev, y, "y", T, H, yt)
    kind, pg, ldg = _gate(fn, dev, gate, "gate", T, H, yt)
    po, ldo = _rows(fn, dev, x_out, "x_out", T, H, x.dtype)
    pn, ldn = _rows(fn, dev, n_out, "n_out", T, H, yt)
    _issue(fn, dev, stream, (px, ldx, xty, py, ldy, yty, pg, kind, ldg, _flat(fn, dev, gamma_post, "gamma_post", (H,)),
                             _flat(fn, dev, gamma_pre, "gamma_pre", (H,)), post_norm and y is not None, scale, eps, T,
                             H, po, ldo, pn, ldn, _flat(fn, dev, rstd_post, "rstd_post", (T,)),
                             _flat(fn, dev, rstd_pre, "rstd_pre", (T,))))


def moe_block_norm_workspace_size(T, H):
    return load().moe_block_norm_workspace_size(T, H)


def moe_block_norm_backward(dx_out, dn, x_out, y, dx, dy, workspace, gamma_post=None, gamma_pre=None, gate=None,
                            scale=1.0, post_norm=True, rstd_post=None, rstd_pre=None, dgate=None, dgamma_post=None,
                            dgamma_pre=None, stream=None):
    """Gradients of moe_block_norm for dx_out (of x_out) and dn (of n_out); either may be None.

    x_out, rstd_post and rstd_pre are what the forward call wrote.  dgate has
    gate's shape and type; dgate, dgamma_post and dgamma_pre may be None.
    """
    fn = "moe_block_norm_backward"
    T, H, xty, dev = _matrix(fn, dx, "dx")
    act = y if y is not None else dn
    if act is None:
        _no(fn, MOE_EINVAL, "y and dn are both None")
    xt, yty, yt = dx.dtype, _type(fn, act, "y" if y is not None else "dn"), act.dtype
    pdo, lddo = _rows(fn, dev, dx_out, "dx_out", T, H, xt)
    pdn, lddn = _rows(fn, dev, dn, "dn", T, H, yt)
    px, ldx = _rows(fn, dev, x_out, "x_out", T, H, xt)
    py, ldy = _rows(fn, dev, y, "y", T, H, yt)
    kind, pg, ldg = _gate(fn, dev, gate, "gate", T, H, yt)
    pdx, lddx = _rows(fn, dev, dx, "dx", T, H, xt)
    pdy, lddy = _rows(fn, dev, dy, "dy", T, H, yt)
    if dgate is not None and gate is None:
        _no(fn, MOE_EINVAL, "dgate without gate")
    _, pdg, lddg = _gate(fn, dev, dgate, "dgate", T, H, yt, kind)
    ws, nbytes = _bytes(fn, dev, workspace, "workspace")
    _issue(fn, dev, stream,
           (pdo, lddo, pdn, lddn, px, ldx, xty, py, ldy, yty, pg, kind, ldg,
            _flat(fn, dev, gamma_post, "gamma_post", (H,)), _flat(fn, dev, gamma_pre, "gamma_pre", (H,)),
            post_norm and y is not None, scale, _flat(fn, dev, rstd_post, "rstd_post", (T,)),
            _flat(fn, dev, rstd_pre, "rstd_pre", (T,)), T, H, pdx, lddx, pdy, lddy, pdg, lddg,
            _flat(fn, dev, dgamma_post, "dgamma_post", (H,)), _flat(fn, dev, dgamma_pre, "dgamma_pre", (H,)), ws, nbytes))


def moe_route_backward_workspace_size(T, k, E, H):
    return load().moe_route_backward_workspace_size(T, k, E, H)


def moe_route_backward(dw, topk_w, topk_ids, x, w_router, offsets, perm, dlogits, dx, dw_router, dbias, workspace,
                       add=None, dev_status=None, stream=None):
    """Gradient of moe_route: from the gradient of the top-k weights to the
    selected logits (dlogits), the tokens (dx, plus add), the router matrix
    and its bias.  dx, dw_router and dbias may be None."""
    fn = "moe_route_backward"
    i32 = torch.int32
    T, H, _, dev = _matrix(fn, x, "x")
    E = len(w_router)
    k, ids = _routes(fn, dev, topk_ids, T, "topk_ids")
    px, ldx = _rows(fn, dev, x, "x", T, H, torch.bfloat16)
    pr, ldr = _rows(fn, dev, w_router, "w_router", E, H, torch.bfloat16)
    dty, pd, ldd, pa, lda = MOE_ROW_F32, None, 0, None, 0
    if dx is not None:
        dty = _type(fn, dx, "dx")
        pd, ldd = _rows(fn, dev, dx, "dx", T, H, dx.dtype)
        pa, lda = _rows(fn, dev, add, "add", T, H, dx.dtype)
    elif add is not None:
        _no(fn, MOE_EINVAL, "add without dx")
    pw, ldw = _rows(fn, dev, dw_router, "dw_router", E, H, torch.float32)
    ws, nbytes = _bytes(fn, dev, workspace, "workspace")
    _issue(fn, dev, stream,
           (_flat(fn, dev, dw, "dw", (T, k)), _flat(fn, dev, topk_w, "topk_w", (T, k)), ids, px, ldx, pr, ldr,
            _flat(fn, dev, offsets, "offsets", (E + 1,), i32), _flat(fn, dev, perm, "perm", (T * k,), i32), T, k, E, H,
            _flat(fn, dev, dlogits, "dlogits", (T, k)), pd, ldd, dty, pa, lda, pw, ldw,
            _flat(fn, dev, dbias, "dbias", (E,)), ws, nbytes, _flat(fn, dev, dev_status, "dev_status", (1,), i32)))
