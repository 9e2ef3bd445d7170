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
from ._lib import MOE_EINVAL, MOE_ESHAPE, MOE_OK, MoEError

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
        _build.build()
        lib = C.CDLL(_build.LIB_BLOCK)
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


class _Call:
    """The checks of one call: every tensor on one GPU, of the shape asked."""

    __slots__ = ("fn", "dev")

    def __init__(self, fn, t):
        self.fn = fn
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise MoEError(fn, MOE_EINVAL, "tensors must be on a GPU")
        self.dev = t.get_device()

    def no(self, status, what):
        raise MoEError(self.fn, status, what)

    def _tensor(self, t, name):
        if not isinstance(t, torch.Tensor) or t.get_device() != self.dev:
            self.no(MOE_EINVAL, f"{name} is not a tensor on GPU {self.dev}")

    def rows(self, t, name, n, H, dtype=None):
        """(pointer, row stride) of a [n, H] matrix; (None, 0) for None."""
        if t is None:
            return None, 0
        self._tensor(t, name)
        if tuple(t.shape) != (n, H):
            self.no(MOE_ESHAPE, f"{name} has shape {tuple(t.shape)}, expected {(n, H)}")
        if t.dtype not in _TYPES if dtype is None else t.dtype != dtype:
            self.no(MOE_EINVAL, f"{name} has type {t.dtype}, expected {dtype or 'float32 or bfloat16'}")
        ld, step = t.stride()
        if step != 1 and H > 1:
            self.no(MOE_EINVAL, f"{name}: the elements of a row must be adjacent")
        return t.data_ptr(), ld if n > 1 else max(ld, H)

    def flat(self, t, name, shape, dtype=torch.float32):
        """Pointer of a contiguous array; None for None."""
        if t is None:
            return None
        self._tensor(t, name)
        if tuple(t.shape) != shape:
            self.no(MOE_ESHAPE, f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if t.dtype != dtype:
            self.no(MOE_EINVAL, f"{name} has type {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            self.no(MOE_EINVAL, f"{name} is not contiguous")
        return t.data_ptr()

    def bytes(self, t, name):
        """(pointer, size in bytes) of a workspace; (None, 0) for None."""
        if t is None:
            return None, 0
        self._tensor(t, name)
        if not t.is_contiguous():
            self.no(MOE_EINVAL, f"{name} is not contiguous")
        return t.data_ptr(), t.numel() * t.element_size()

    def matrix(self, t, name):
        """Rows, width and type of the matrix that the others are measured by."""
        self._tensor(t, name)
        if t.dim() != 2:
            self.no(MOE_ESHAPE, f"{name} must be two-dimensional")
        if t.dtype not in _TYPES:
            self.no(MOE_EINVAL, f"{name} has type {t.dtype}, expected float32 or bfloat16")
        return t.shape[0], t.shape[1], _TYPES[t.dtype]

    def issue(self, stream, *args):
        """The C call with the GPU of its tensors current, on `stream` or that GPU's current stream."""
        fn = getattr(load(), self.fn)
        if self.dev == torch.cuda.current_device():
            st = fn(*args, (torch.cuda.current_stream() if stream is None else stream).cuda_stream)
        else:
            with torch.cuda.device(self.dev):
                st = fn(*args, (torch.cuda.current_stream() if stream is None else stream).cuda_stream)
        if st != MOE_OK:
            raise MoEError(self.fn, st, _lib.status_str(st))


def _routes(c, inv_perm, T, name="inv_perm"):
    if not isinstance(inv_perm, torch.Tensor) or inv_perm.dim() != 2:
        c.no(MOE_ESHAPE, f"{name} must be [T, k]")
    k = inv_perm.shape[1]
    return k, c.flat(inv_perm, name, (T, k), torch.int32)


def moe_dispatch(x, inv_perm, x_perm, w=None, dev_status=None, stream=None):
    """x_perm[inv_perm[t,j]] = w[t,j] * x[t] (w None: 1); routes of slot -1 and rows without a route are left out."""
    c = _Call("moe_dispatch", x)
    T, H, ty = c.matrix(x, "x")
    k, inv = _routes(c, inv_perm, T)
    R = c.matrix(x_perm, "x_perm")[0]
    px, ldx = c.rows(x, "x", T, H)
    pp, ldp = c.rows(x_perm, "x_perm", R, H, x.dtype)
    c.issue(stream, px, ldx, ty, inv, c.flat(w, "w", (T, k)), T, k, H, R, pp, ldp,
            c.flat(dev_status, "dev_status", (1,), torch.int32))


def moe_dispatch_backward(dx_perm, inv_perm, dx, w=None, x=None, dw=None, add=None, dev_status=None, stream=None):
    """dx = add + sum_j w * dx_perm[inv_perm]; with dw (and x), dw[t,j] = <dx_perm[inv_perm[t,j]], x[t]>."""
    c = _Call("moe_dispatch_backward", dx)
    T, H, dty = c.matrix(dx, "dx")
    k, inv = _routes(c, inv_perm, T)
    R, _, ty = c.matrix(dx_perm, "dx_perm")
    pp, ldp = c.rows(dx_perm, "dx_perm", R, H)
    px, ldx = c.rows(x, "x", T, H, dx_perm.dtype)
    pd, ldd = c.rows(dx, "dx", T, H)
    pa, lda = c.rows(add, "add", T, H, dx.dtype)
    c.issue(stream, pp, ldp, ty, inv, c.flat(w, "w", (T, k)), px, ldx, T, k, H, R, pd, ldd, dty, pa, lda,
            c.flat(dw, "dw", (T, k)), c.flat(dev_status, "dev_status", (1,), torch.int32))


def moe_collect(y_perm, inv_perm, w, out, add=None, dev_status=None, stream=None):
    """out = add + sum_j w * y_perm[inv_perm] in rank order (w None: 1)."""
    c = _Call("moe_collect", out)
    T, H, oty = c.matrix(out, "out")
    k, inv = _routes(c, inv_perm, T)
    R, _, ty = c.matrix(y_perm, "y_perm")
    pp, ldp = c.rows(y_perm, "y_perm", R, H)
    po, ldo = c.rows(out, "out", T, H)
    pa, lda = c.rows(add, "add", T, H, out.dtype)
    c.issue(stream, pp, ldp, ty, inv, c.flat(w, "w", (T, k)), T, k, H, R, po, ldo, oty, pa, lda,
            c.flat(dev_status, "dev_status", (1,), torch.int32))


def moe_collect_backward(dout, y_perm, inv_perm, w, dy_perm, dw=None, dev_status=None, stream=None):
    """dy_perm[inv_perm[t,j]] = w[t,j] * dout[t]; with dw (and y_perm), dw[t,j] = <dout[t], y_perm[inv_perm[t,j]]>."""
    c = _Call("moe_collect_backward", dout)
    T, H, oty = c.matrix(dout, "dout")
    k, inv = _routes(c, inv_perm, T)
    R, _, ty = c.matrix(dy_perm, "dy_perm")
    po, ldo = c.rows(dout, "dout", T, H)
    py, ldy = c.rows(y_perm, "y_perm", R, H, dy_perm.dtype)
    pd, ldd = c.rows(dy_perm, "dy_perm", R, H)
    c.issue(stream, po, ldo, oty, py, ldy, ty, inv, c.flat(w, "w", (T, k)), T, k, H, R, pd, ldd,
            c.flat(dw, "dw", (T, k)), c.flat(dev_status, "dev_status", (1,), torch.int32))


def _gate(c, gate, name, T, H, dtype, kind=None):
    """(kind, pointer, row stride): [H] per channel, [T, 1] per token, [T, H] elementwise (of y's type)."""
    if gate is None:
        return MOE_GATE_NONE, None, 0
    if not isinstance(gate, torch.Tensor):
        c.no(MOE_EINVAL, f"{name} is not a tensor on GPU {c.dev}")
    if kind is None:
        if gate.dim() == 1:
            kind = MOE_GATE_CHANNEL
        else:
            kind = MOE_GATE_TOKEN if gate.dim() == 2 and gate.shape[1] == 1 and gate.dtype == torch.float32 \
                else MOE_GATE_FULL
    if kind == MOE_GATE_CHANNEL:
        return kind, c.flat(gate, name, (H,)), 0
    if kind == MOE_GATE_TOKEN:
        return kind, c.flat(gate, name, (T, 1)), 0
    return (kind,) + c.rows(gate, name, T, H, dtype)


def moe_block_norm(x, y, x_out, n_out, gamma_post=None, gamma_pre=None, gate=None, scale=1.0, eps=1e-6,
                   post_norm=True, rstd_post=None, rstd_pre=None, stream=None):
    """x_out = scale * x + gate * RMSNorm(y), n_out = RMSNorm(x_out), in one pass.

    y None: no block before it (x_out = scale * x); x_out or n_out None: not
    wanted.  gate: [H], [T, 1] (both fp32) or [T, H] of y's type.  The norms'
    gain is 1 + gamma; post_norm=False leaves y as it is.
    """
    c = _Call("moe_block_norm", x)
    T, H, xty = c.matrix(x, "x")
    act = y if y is not None else n_out
    if act is None:
        c.no(MOE_EINVAL, "y and n_out are both None")
    yty = c.matrix(act, "y" if y is not None else "n_out")[2]
    post_norm = bool(post_norm) and y is not None
    px, ldx = c.rows(x, "x", T, H)
    py, ldy = c.rows(y, "y", T, H)
    kind, pg, ldg = _gate(c, gate, "gate", T, H, act.dtype)
    po, ldo = c.rows(x_out, "x_out", T, H, x.dtype)
    pn, ldn = c.rows(n_out, "n_out", T, H, act.dtype)
    c.issue(stream, px, ldx, xty, py, ldy, yty, pg, kind, ldg, c.flat(gamma_post, "gamma_post", (H,)),
            c.flat(gamma_pre, "gamma_pre", (H,)), post_norm, scale, eps, T, H, po, ldo, pn, ldn,
            c.flat(rstd_post, "rstd_post", (T,)), c.flat(rstd_pre, "rstd_pre", (T,)))


def moe_block_norm_workspace_size(T, H):
    return load().moe_block_norm_workspace_size(T, H)


def moe_block_norm_backward(dx_out, dn, x_out, y, dx, dy, workspace, gamma_post=None, gamma_pre=None, gate=None,
                            scale=1.0, post_norm=True, rstd_post=None, rstd_pre=None, dgate=None, dgamma_post=None,
                            dgamma_pre=None, stream=None):
    """Gradients of moe_block_norm for dx_out (of x_out) and dn (of n_out); either may be None.

    x_out, rstd_post and rstd_pre are what the forward call wrote.  dgate has
    gate's shape and type; dgate, dgamma_post and dgamma_pre may be None.
    """
    c = _Call("moe_block_norm_backward", dx)
    T, H, xty = c.matrix(dx, "dx")
    act = y if y is not None else dn
    if act is None:
        c.no(MOE_EINVAL, "y and dn are both None")
    yty = c.matrix(act, "y" if y is not None else "dn")[2]
    post_norm = bool(post_norm) and y is not None
    pdo, lddo = c.rows(dx_out, "dx_out", T, H, dx.dtype)
    pdn, lddn = c.rows(dn, "dn", T, H, act.dtype)
    px, ldx = c.rows(x_out, "x_out", T, H, dx.dtype)
    py, ldy = c.rows(y, "y", T, H)
    kind, pg, ldg = _gate(c, gate, "gate", T, H, act.dtype)
    pdx, lddx = c.rows(dx, "dx", T, H)
    pdy, lddy = c.rows(dy, "dy", T, H, act.dtype)
    if dgate is not None and gate is None:
        c.no(MOE_EINVAL, "dgate without gate")
    _, pdg, lddg = _gate(c, dgate, "dgate", T, H, act.dtype, kind)
    ws, nbytes = c.bytes(workspace, "workspace")
    c.issue(stream, pdo, lddo, pdn, lddn, px, ldx, xty, py, ldy, yty, pg, kind, ldg,
            c.flat(gamma_post, "gamma_post", (H,)), c.flat(gamma_pre, "gamma_pre", (H,)), post_norm, scale,
            c.flat(rstd_post, "rstd_post", (T,)), c.flat(rstd_pre, "rstd_pre", (T,)), T, H, pdx, lddx, pdy, lddy,
            pdg, lddg, c.flat(dgamma_post, "dgamma_post", (H,)), c.flat(dgamma_pre, "dgamma_pre", (H,)), ws, nbytes)


def moe_route_backward_workspace_size(T, k, E, H):
    return load().moe_route_backward_workspace_size(T, k, E, H)


def moe_route_backward(dw, topk_w, topk_ids, x, w_router, offsets, perm, dlogits, dx, dw_router, dbias, workspace,
                       add=None, dev_status=None, stream=None):
    """Gradient of moe_route: from the gradient of the top-k weights to the
    selected logits (dlogits), the tokens (dx, plus add), the router matrix
    and its bias.  dx, dw_router and dbias may be None."""
    c = _Call("moe_route_backward", x)
    T, H, _ = c.matrix(x, "x")
    E = c.matrix(w_router, "w_router")[0]
    k, ids = _routes(c, topk_ids, T, "topk_ids")
    px, ldx = c.rows(x, "x", T, H, torch.bfloat16)
    pr, ldr = c.rows(w_router, "w_router", E, H, torch.bfloat16)
    dty = MOE_ROW_F32 if dx is None else c.matrix(dx, "dx")[2]
    pd, ldd = c.rows(dx, "dx", T, H)
    if add is not None and dx is None:
        c.no(MOE_EINVAL, "add without dx")
    pa, lda = c.rows(add, "add", T, H, None if dx is None else dx.dtype)
    pw, ldw = c.rows(dw_router, "dw_router", E, H, torch.float32)
    ws, nbytes = c.bytes(workspace, "workspace")
    c.issue(stream, c.flat(dw, "dw", (T, k)), c.flat(topk_w, "topk_w", (T, k)), ids, px, ldx, pr, ldr,
            c.flat(offsets, "offsets", (E + 1,), torch.int32), c.flat(perm, "perm", (T * k,), torch.int32), T, k, E, H,
            c.flat(dlogits, "dlogits", (T, k)), pd, ldd, dty, pa, lda, pw, ldw, c.flat(dbias, "dbias", (E,)), ws, nbytes,
            c.flat(dev_status, "dev_status", (1,), torch.int32))
