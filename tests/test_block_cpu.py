"""Host side of libmoe_block without a GPU: exports, refusals, and the
reference gradients of the GPU tests against differences of the definitions."""
import ctypes as C
import subprocess

import pytest
import torch

import block_reference as ref
from sparse_moe_routed_gb300 import MoEError, _block, _lib

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: CPU-only host checks")

A = [C.c_void_p((1 << 20) + (i << 16)) for i in range(24)]  # 64 KB apart, aligned placeholders
ODD = C.c_void_p((1 << 20) + 1)
F32, BF16 = _block.MOE_ROW_F32, _block.MOE_ROW_BF16


def test_exports_match_header_exactly():
    L = _block.load()
    text = subprocess.run(["nm", "-D", "--defined-only", _block._build.LIB_BLOCK], capture_output=True, text=True).stdout
    assert sorted(x.split()[-1] for x in text.splitlines() if " T " in x) == _block.declared_functions()
    assert L.moe_block_abi_version() == 100


def _status(name, spec, kw):
    unknown = set(kw) - {k for k, _ in spec}
    assert not unknown, unknown
    return getattr(_block.load(), name)(*[kw.get(k, v) for k, v in spec])


DISPATCH = [("x", A[0]), ("ldx", 64), ("type", BF16), ("inv", A[1]), ("w", A[2]), ("T", 16), ("k", 4), ("H", 64),
            ("R", 64), ("xp", A[3]), ("ldp", 64), ("status", None), ("stream", None)]
DISPATCH_B = [("dxp", A[0]), ("ldp", 64), ("type", BF16), ("inv", A[1]), ("w", A[2]), ("x", A[3]), ("ldx", 64),
              ("T", 16), ("k", 4), ("H", 64), ("R", 64), ("dx", A[4]), ("ldd", 64), ("dtype", F32), ("add", A[5]),
              ("lda", 64), ("dw", A[6]), ("status", None), ("stream", None)]
COLLECT = [("yp", A[0]), ("ldp", 64), ("type", BF16), ("inv", A[1]), ("w", A[2]), ("T", 16), ("k", 4), ("H", 64),
           ("R", 64), ("out", A[3]), ("ldo", 64), ("otype", F32), ("add", None), ("lda", 0), ("status", None),
           ("stream", None)]
COLLECT_B = [("dout", A[0]), ("ldo", 64), ("otype", F32), ("yp", A[1]), ("ldp", 64), ("type", BF16), ("inv", A[2]),
             ("w", A[3]), ("T", 16), ("k", 4), ("H", 64), ("R", 64), ("dyp", A[4]), ("ldd", 64), ("dw", A[5]),
             ("status", None), ("stream", None)]
NORM = [("x", A[0]), ("ldx", 64), ("xtype", F32), ("y", A[1]), ("ldy", 64), ("ytype", BF16), ("gate", A[2]),
        ("kind", _block.MOE_GATE_CHANNEL), ("ldg", 0), ("gpost", A[3]), ("gpre", A[4]), ("post", 1), ("scale", 1.0),
        ("eps", 1e-6), ("T", 16), ("H", 64), ("xo", A[5]), ("ldxo", 64), ("n", A[6]), ("ldn", 64), ("r1", A[7]),
        ("r2", A[8]), ("stream", None)]
NORM_B = [("dxo", A[0]), ("lddxo", 64), ("dn", A[1]), ("lddn", 64), ("xo", A[2]), ("ldxo", 64), ("xtype", F32),
          ("y", A[3]), ("ldy", 64), ("ytype", BF16), ("gate", A[4]), ("kind", _block.MOE_GATE_CHANNEL), ("ldg", 0),
          ("gpost", A[5]), ("gpre", A[6]), ("post", 1), ("scale", 1.0), ("r1", A[7]), ("r2", A[8]), ("T", 16),
          ("H", 64), ("dx", A[9]), ("lddx", 64), ("dy", A[10]), ("lddy", 64), ("dgate", A[11]), ("lddg", 0),
          ("dgpost", A[12]), ("dgpre", A[13]), ("ws", A[14]), ("wsb", 1 << 24), ("stream", None)]
ROUTE_B = [("dw", A[0]), ("w", A[1]), ("ids", A[2]), ("x", A[3]), ("ldx", 64), ("wr", A[4]), ("ldr", 64),
           ("offsets", A[5]), ("perm", A[6]), ("T", 16), ("k", 4), ("E", 8), ("H", 64), ("dl", A[7]), ("dx", A[8]),
           ("ldd", 64), ("dtype", F32), ("add", None), ("lda", 0), ("dwr", A[9]), ("lddw", 64), ("db", A[10]),
           ("ws", A[11]), ("wsb", 1 << 20), ("status", None), ("stream", None)]

CALLS = {"moe_dispatch": DISPATCH, "moe_dispatch_backward": DISPATCH_B, "moe_collect": COLLECT,
         "moe_collect_backward": COLLECT_B, "moe_block_norm": NORM, "moe_block_norm_backward": NORM_B,
         "moe_route_backward": ROUTE_B}
EINVAL, ESHAPE, ENOTSUP, EWS = _lib.MOE_EINVAL, _lib.MOE_ESHAPE, _lib.MOE_ENOTSUP, _lib.MOE_EWORKSPACE

REFUSALS = [
    ("moe_dispatch", dict(x=None), EINVAL), ("moe_dispatch", dict(inv=None), EINVAL),
    ("moe_dispatch", dict(xp=None), EINVAL), ("moe_dispatch", dict(xp=A[0]), EINVAL),
    ("moe_dispatch", dict(type=2), EINVAL), ("moe_dispatch", dict(x=ODD), EINVAL), ("moe_dispatch", dict(w=ODD), EINVAL),
    ("moe_dispatch", dict(T=-1), ESHAPE), ("moe_dispatch", dict(k=0), ESHAPE), ("moe_dispatch", dict(H=0), ESHAPE),
    ("moe_dispatch", dict(R=-1), ESHAPE), ("moe_dispatch", dict(ldx=63), ESHAPE), ("moe_dispatch", dict(ldp=0), ESHAPE),
    ("moe_dispatch", dict(ldx=-64), ESHAPE), ("moe_dispatch", dict(k=33), ENOTSUP),
    ("moe_dispatch", dict(H=65537, ldx=1 << 17, ldp=1 << 17), ENOTSUP), ("moe_dispatch", dict(T=1 << 29), ENOTSUP),
    ("moe_dispatch", dict(ldx=1 << 60), ENOTSUP), ("moe_dispatch", dict(T=(1 << 30) + 1, k=1), ENOTSUP),
    ("moe_block_norm", dict(T=(1 << 30) + 1), ENOTSUP), ("moe_route_backward", dict(T=(1 << 30) + 1, k=1), ENOTSUP),
    ("moe_dispatch_backward", dict(dxp=None), EINVAL), ("moe_dispatch_backward", dict(dx=None), EINVAL),
    ("moe_dispatch_backward", dict(x=None), EINVAL), ("moe_dispatch_backward", dict(dx=A[0]), EINVAL),
    ("moe_dispatch_backward", dict(dx=A[3]), EINVAL), ("moe_dispatch_backward", dict(add=A[4], lda=128), EINVAL),
    ("moe_dispatch_backward", dict(dtype=-1), EINVAL), ("moe_dispatch_backward", dict(lda=1), ESHAPE),
    ("moe_collect", dict(yp=None), EINVAL), ("moe_collect", dict(out=None), EINVAL),
    ("moe_collect", dict(out=A[0]), EINVAL), ("moe_collect", dict(ldo=8), ESHAPE), ("moe_collect", dict(otype=7), EINVAL),
    ("moe_collect_backward", dict(dout=None), EINVAL), ("moe_collect_backward", dict(yp=None), EINVAL),
    ("moe_collect_backward", dict(dyp=A[1]), EINVAL), ("moe_collect_backward", dict(dyp=None), EINVAL),
    ("moe_collect_backward", dict(ldd=63), ESHAPE),
    ("moe_block_norm", dict(x=None), EINVAL), ("moe_block_norm", dict(y=None), EINVAL),
    ("moe_block_norm", dict(xo=None, n=None, gpre=None, r2=None), EINVAL), ("moe_block_norm", dict(n=None), EINVAL),
    ("moe_block_norm", dict(kind=4), EINVAL), ("moe_block_norm", dict(gate=None), EINVAL),
    ("moe_block_norm", dict(kind=0), EINVAL), ("moe_block_norm", dict(post=0), EINVAL),
    ("moe_block_norm", dict(post=0, gpost=None), EINVAL),
    ("moe_block_norm", dict(eps=-1.0), EINVAL), ("moe_block_norm", dict(eps=float("nan")), EINVAL),
    ("moe_block_norm", dict(scale=float("inf")), EINVAL), ("moe_block_norm", dict(xo=A[0], ldxo=72), EINVAL),
    ("moe_block_norm", dict(xo=A[1]), EINVAL), ("moe_block_norm", dict(n=A[1]), EINVAL),
    ("moe_block_norm", dict(H=16385), ENOTSUP), ("moe_block_norm", dict(ldn=63), ESHAPE),
    ("moe_block_norm", dict(kind=3, ldg=1), ESHAPE), ("moe_block_norm", dict(gpre=ODD), EINVAL),
    ("moe_block_norm_backward", dict(dxo=None, dn=None), EINVAL), ("moe_block_norm_backward", dict(dx=None), EINVAL),
    ("moe_block_norm_backward", dict(dy=None), EINVAL), ("moe_block_norm_backward", dict(xo=None), EINVAL),
    ("moe_block_norm_backward", dict(r1=None), EINVAL), ("moe_block_norm_backward", dict(r2=None), EINVAL),
    ("moe_block_norm_backward", dict(kind=0, gate=None), EINVAL), ("moe_block_norm_backward", dict(dy=A[3]), EINVAL),
    ("moe_block_norm_backward", dict(dx=A[0], lddx=72), EINVAL), ("moe_block_norm_backward", dict(dx=A[2]), EINVAL),
    ("moe_block_norm_backward", dict(ws=None), EWS), ("moe_block_norm_backward", dict(wsb=16), EWS),
    ("moe_block_norm_backward", dict(ws=ODD), EINVAL), ("moe_block_norm_backward", dict(lddy=0), ESHAPE),
    ("moe_route_backward", dict(dw=None), EINVAL), ("moe_route_backward", dict(dl=None), EINVAL),
    ("moe_route_backward", dict(dl=A[0]), EINVAL), ("moe_route_backward", dict(wr=None), EINVAL),
    ("moe_route_backward", dict(x=None), EINVAL), ("moe_route_backward", dict(perm=None), EINVAL),
    ("moe_route_backward", dict(offsets=None), EINVAL), ("moe_route_backward", dict(ws=None), EWS),
    ("moe_route_backward", dict(wsb=8), EWS), ("moe_route_backward", dict(ws=ODD), EINVAL),
    ("moe_route_backward", dict(k=9), ENOTSUP), ("moe_route_backward", dict(E=1025), ENOTSUP),
    ("moe_route_backward", dict(ldr=8), ESHAPE), ("moe_route_backward", dict(E=0), ESHAPE),
    ("moe_route_backward", dict(add=A[8], lda=72), EINVAL), ("moe_route_backward", dict(dx=A[3]), EINVAL),
]


@no_gpu
@pytest.mark.parametrize("name,kw,code", REFUSALS, ids=lambda v: v if isinstance(v, str) else None)
def test_refusals(name, kw, code):
    assert _status(name, CALLS[name], kw) == code


@no_gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_arguments_are_admitted(name):
    """The unchanged arguments pass the host checks (and reach the device, absent here)."""
    assert _status(name, CALLS[name], {}) == _lib.MOE_ECUDA


@no_gpu
@pytest.mark.parametrize("name,kw", [
    ("moe_dispatch", dict(w=None)), ("moe_dispatch", dict(k=32, R=512)), ("moe_dispatch", dict(H=65536, ldx=65536, ldp=65536)),
    ("moe_dispatch_backward", dict(dw=None, x=None)), ("moe_dispatch_backward", dict(add=A[4])),
    ("moe_collect", dict(add=A[3], lda=64)), ("moe_collect_backward", dict(dw=None, yp=None)),
    ("moe_block_norm", dict(xo=A[0])), ("moe_block_norm", dict(xo=None)),
    ("moe_block_norm", dict(n=None, gpre=None, r2=None)),
    ("moe_block_norm", dict(y=None, gate=None, kind=0, gpost=None, post=0, r1=None)),
    ("moe_block_norm", dict(H=16384, ldx=16384, ldy=16384, ldxo=16384, ldn=16384)),
    ("moe_block_norm_backward", dict(dx=A[0])), ("moe_block_norm_backward", dict(dxo=None)),
    ("moe_block_norm_backward", dict(dn=None, xo=None, r2=None, gpre=None, dgpre=None)),
    ("moe_block_norm_backward", dict(dgate=None, dgpost=None, dgpre=None, ws=None, wsb=0)),
    ("moe_route_backward", dict(dx=None)), ("moe_route_backward", dict(dwr=None, db=None, ws=None, wsb=0)),
    ("moe_route_backward", dict(add=A[8], lda=64)),
])
def test_optional_arguments_are_admitted(name, kw):
    assert _status(name, CALLS[name], kw) == _lib.MOE_ECUDA


@no_gpu
@pytest.mark.parametrize("name,empty", [
    ("moe_dispatch", ("x", "inv", "w")), ("moe_dispatch_backward", ("x", "inv", "w", "dx", "add", "dw")),
    ("moe_collect", ("inv", "w", "out")), ("moe_collect_backward", ("dout", "inv", "w", "dw")),
    ("moe_block_norm", ("x", "y", "xo", "n", "r1", "r2"))])
def test_no_tokens_is_accepted_with_null_arrays(name, empty):
    assert _status(name, CALLS[name], dict(T=0, **{n: None for n in empty})) == _lib.MOE_OK


def test_workspace_sizes():
    L = _block.load()
    assert L.moe_block_norm_workspace_size(-1, 64) == 0
    assert L.moe_block_norm_workspace_size(4, 0) == 0
    assert L.moe_block_norm_workspace_size(4, 16385) == 0
    assert L.moe_block_norm_workspace_size(0, 64) > 0
    assert L.moe_block_norm_workspace_size(1 << 20, 16384) >= L.moe_block_norm_workspace_size(1, 16384) > 0
    assert L.moe_route_backward_workspace_size(16, 33, 64, 64) == 0
    assert L.moe_route_backward_workspace_size(16, 4, 1025, 64) == 0
    assert L.moe_route_backward_workspace_size(0, 4, 64, 64) > 0
    # large route counts do not wrap
    assert L.moe_route_backward_workspace_size(1 << 25, 32, 1024, 65536) > 1 << 40


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 64))
    inv = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(MoEError) as e:
        _block.moe_dispatch(x, inv, torch.zeros((8, 64)))
    assert e.value.status == EINVAL
    with pytest.raises(MoEError):
        _block.moe_block_norm(x, x, x, x)


# -- the reference gradients against differences of the definitions ----------
def _diff(f, v, h=1e-6):
    """Central differences of the scalar f with respect to the tensor v (float64)."""
    g = torch.zeros_like(v)
    flat, out = v.view(-1), g.view(-1)
    for i in range(v.numel()):
        keep = float(flat[i])
        flat[i] = keep + h
        a = f()
        flat[i] = keep - h
        b = f()
        flat[i] = keep
        out[i] = (a - b) / (2 * h)
    return g


# a central difference of a smooth f is off by h^2 |f'''| / 6 (1e-12 scale) and
# 2^-53 |f| / h (1e-9 scale here): 1e-7 of the largest entry holds both
def _near(a, b):
    assert float((a - b).abs().max()) <= 1e-7 * max(1.0, float(b.abs().max()))


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_norm_gradient_formula_against_differences(gate, post):
    g = torch.Generator().manual_seed(7)
    T, H, scale, eps = 3, 5, 0.75, 1e-3
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, y, gp, gq = rnd(T, H), rnd(T, H), 0.1 * rnd(H), 0.1 * rnd(H)
    gt = {"none": None, "channel": rnd(H), "token": rnd(T, 1), "full": rnd(T, H)}[gate]
    a, b = rnd(T, H), rnd(T, H)
    args = lambda: (x, y, gt, gp if post else None, gq, scale, eps, post, torch.float64, torch.float64)

    def loss():
        f = ref.norm(*args())
        return float((a * f["x_out"][0]).sum() + (b * f["n_out"][0]).sum())

    f = ref.norm(*args())
    r1 = ref.rstd(y, eps)[0][:, 0]
    r2 = ref.rstd(f["x_out"][0], eps)[0][:, 0]
    got = ref.norm_grad(a, b, f["x_out"][0], y, gt, gp if post else None, gq, scale, r1, r2, post, torch.float64,
                        torch.float64)
    _near(got["dx"][0], _diff(loss, x))
    _near(got["dy"][0], _diff(loss, y))
    _near(got["dgamma_pre"][0], _diff(loss, gq))
    if post:
        _near(got["dgamma_post"][0], _diff(loss, gp))
    if gt is not None:
        _near(got["dgate"][0], _diff(loss, gt))


def test_row_gradient_formulas_against_differences():
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    T, H, k, R = 3, 4, 2, 7
    inv = torch.tensor([[3, 0], [-1, 6], [1, -1]], dtype=torch.int32)
    x, w, y, a, b, add = rnd(T, H), rnd(T, k), rnd(R, H), rnd(R, H), rnd(T, H), rnd(T, H)
    zero = torch.zeros(R, H, dtype=torch.float64)
    f8 = torch.float64
    disp = lambda: float((a * ref.spread(x, inv, w, zero)[0]).sum())
    # dispatch's gradient for the gradient `a` of its rows
    _near(ref.join(a, inv, w, None, f8)[0], _diff(disp, x))
    _near(ref.dots(a, inv, x)[0], _diff(disp, w))
    coll = lambda: float((b * ref.join(y, inv, w, add, f8)[0]).sum())
    _near(ref.spread(b, inv, w, zero)[0], _diff(coll, y))
    _near(ref.dots(y, inv, b)[0], _diff(coll, w))


def test_route_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    T, H, E, k = 3, 4, 6, 3
    x, wr, bias, a = rnd(T, H), rnd(E, H), rnd(E), rnd(T, k)
    ids = (x @ wr.t() + bias).topk(k, dim=1)[1]
    weights = lambda: torch.softmax((x @ wr.t() + bias).gather(1, ids), dim=1)
    f = lambda: float((a * weights()).sum())
    got = ref.route_grad(a, weights(), ids, x, wr, None, torch.float64)
    _near(got["dx"][0], _diff(f, x))
    _near(got["dw_router"][0], _diff(f, wr))
    _near(got["dbias"][0], _diff(f, bias))
