"""libmoe_block on the GPU against its definitions in 64 bits.

Every output is compared element by element with block_reference.py, inside
the bound that goes with it there.
"""
import pytest
import torch

import block_reference as ref
import sparse_moe_routed_gb300 as M
from sparse_moe_routed_gb300 import MoEError, _block, _lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)]
NAN = float("nan")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def view(n, H, dtype, pad=0, shift=0, fill=-7.0):
    """[n, H] rows, `pad` columns apart, the first `shift` elements into the buffer; with the whole buffer."""
    buf = torch.full((n * (H + pad) + shift + 8,), fill, dtype=dtype, device=DEV)
    return torch.as_strided(buf, (n, H), (H + pad, 1), shift), buf


def rand(g, n, H, dtype, pad=0, shift=0, std=1.0):
    v, _ = view(n, H, dtype, pad, shift)
    v.copy_(torch.randn((n, H), generator=g, device=DEV) * std)
    return v


def near(got, want, name=""):
    value, bound = want
    off = (got.to(torch.float64) - value).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst {float((off - bound).max()):.3e}"


def untouched(buf, v, fill=-7.0):
    """Everything in v's buffer outside v still holds the fill."""
    mask = torch.ones(buf.shape, dtype=torch.bool, device=DEV)
    torch.as_strided(mask, v.shape, v.stride(), v.storage_offset()).fill_(False)
    assert bool((buf[mask] == fill).all())


def routes(g, T, k, R=None, drop=0.0):
    """Distinct slots for T*k routes among R >= T*k, some without one."""
    R = T * k if R is None else R
    inv = torch.randperm(R, generator=g, device=DEV)[:T * k].to(torch.int32).view(T, k)
    if drop:
        inv = torch.where(torch.rand((T, k), generator=g, device=DEV) < drop, torch.full_like(inv, -1), inv)
    return inv.contiguous()


SIZES = [  # T, H, k
    (1, 1, 1), (1, 7, 2), (3, 8, 1), (2, 255, 5), (5, 256, 8), (1, 2560, 10), (16, 2560, 10), (17, 257, 9),
    (33, 1001, 16), (9, 520, 17), (4, 264, 32), (700, 64, 6), (1300, 136, 10), (2, 16400, 3), (1, 65536, 2),
]


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("T,H,k", SIZES)
@pytest.mark.parametrize("pad,shift,drop", [(0, 0, 0.0), (8, 0, 0.3), (3, 1, 0.3), (2, 2, 0.0)])
def test_rows_to_experts_and_back(T, H, k, types, pad, shift, drop):
    rows, tok = types
    g = gen(T * 7919 + H * 31 + k)
    R = T * k + 3
    inv = routes(g, T, k, R, drop)
    w = torch.randn((T, k), generator=g, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    free = torch.ones(R, dtype=torch.bool, device=DEV)
    free[inv[inv >= 0].long()] = False

    # dispatch, and its gradient
    x = rand(g, T, H, rows, pad, shift)
    for wt in (w, None):
        xp, buf = view(R, H, rows, pad, shift)
        M.moe_dispatch(x, inv, xp, w=wt, dev_status=status)
        near(xp, ref.spread(x, inv, wt, torch.full_like(xp, -7.0)), "x_perm")
        untouched(buf, xp)
    dxp = rand(g, R, H, rows, pad, shift)
    dxp[free] = NAN  # rows that no route names may hold anything
    add = rand(g, T, H, tok, pad, shift)
    dx, buf = view(T, H, tok, pad, shift)
    dw = torch.full((T, k), NAN, device=DEV)
    M.moe_dispatch_backward(dxp, inv, dx, w=w, x=x, dw=dw, add=add, dev_status=status)
    near(dx, ref.join(dxp, inv, w, add, tok), "dx")
    near(dw, ref.dots(dxp, inv, x), "dw")
    untouched(buf, dx)
    dx2, _ = view(T, H, tok, pad, shift)
    M.moe_dispatch_backward(dxp, inv, dx2)
    near(dx2, ref.join(dxp, inv, None, None, tok), "dx, plain")

    # collect, and its gradient
    yp = rand(g, R, H, rows, pad, shift)
    yp[free] = NAN
    out = add.clone() if pad == 0 and shift == 0 else add
    want = ref.join(yp, inv, w, out, tok)
    M.moe_collect(yp, inv, w, out, add=out, dev_status=status)  # in place
    near(out, want, "out")
    dout = rand(g, T, H, tok, pad, shift)
    dyp, buf = view(R, H, rows, pad, shift)
    dw = torch.full((T, k), NAN, device=DEV)
    M.moe_collect_backward(dout, yp, inv, w, dyp, dw, dev_status=status)
    near(dyp, ref.spread(dout, inv, w, torch.full_like(dyp, -7.0)), "dy_perm")
    near(dw, ref.dots(yp, inv, dout), "dw")
    untouched(buf, dyp)
    dyp2, _ = view(R, H, rows, pad, shift)
    M.moe_collect_backward(dout, None, inv, None, dyp2)
    near(dyp2, ref.spread(dout, inv, None, torch.full_like(dyp, -7.0)), "dy_perm, plain")
    assert int(status) == 0


def test_collect_has_the_bits_of_combine():
    g = gen(5)
    T, H, k = 40, 2560, 10
    inv, y = routes(g, T, k), rand(g, T * k, H, F32)
    w, res = torch.rand((T, k), generator=g, device=DEV), rand(g, T, H, F32)
    a, b = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    _lib.moe_combine(y, inv, w, res, None, a, None)
    M.moe_collect(y, inv, w, b, add=res)
    assert torch.equal(a, b)


def test_all_routes_dropped_and_no_slots():
    x = torch.randn((5, 64), device=DEV)
    inv = torch.full((5, 3), -1, dtype=torch.int32, device=DEV)
    none = torch.empty((0, 64), device=DEV)
    M.moe_dispatch(x, inv, none)
    out, dw = torch.full((5, 64), NAN, device=DEV), torch.full((5, 3), NAN, device=DEV)
    M.moe_collect(none, inv, None, out)
    assert bool((out == 0).all())
    M.moe_dispatch_backward(none, inv, out, w=torch.ones((5, 3), device=DEV), x=x, dw=dw, add=x)
    assert torch.equal(out, x) and bool((dw == 0).all())
    dw.fill_(NAN)
    M.moe_collect_backward(x, none, inv, torch.ones((5, 3), device=DEV), none, dw)
    assert bool((dw == 0).all())


def test_no_tokens():
    x, rows = torch.empty((0, 64), device=DEV), torch.full((6, 64), 2.0, device=DEV)
    inv, w = torch.empty((0, 3), dtype=torch.int32, device=DEV), torch.empty((0, 3), device=DEV)
    M.moe_dispatch(x, inv, rows, w=w)
    M.moe_dispatch_backward(rows, inv, x.clone(), w=w, x=x, dw=w.clone())
    M.moe_collect(rows, inv, w, x.clone())
    M.moe_collect_backward(x, rows.clone(), inv, w, rows, w.clone())
    assert bool((rows == 2).all())
    H = 40
    e = lambda *s: torch.empty(s, device=DEV)
    M.moe_block_norm(e(0, H), e(0, H), e(0, H), e(0, H), rstd_post=e(0), rstd_pre=e(0))
    cols = [torch.full((H,), NAN, device=DEV) for _ in range(3)]
    ws = torch.empty(M.moe_block_norm_workspace_size(0, H), dtype=torch.uint8, device=DEV)
    M.moe_block_norm_backward(e(0, H), e(0, H), e(0, H), e(0, H), e(0, H), e(0, H), ws, gate=torch.ones(H, device=DEV),
                              rstd_post=e(0), rstd_pre=e(0), dgate=cols[0], dgamma_post=cols[1], dgamma_pre=cols[2])
    assert all(bool((c == 0).all()) for c in cols)
    E = 9
    dwr, db = torch.full((E, H), NAN, device=DEV), torch.full((E,), NAN, device=DEV)
    xb = torch.empty((0, H), dtype=BF16, device=DEV)
    garbage = torch.full((E + 1,), 77, dtype=torch.int32, device=DEV)  # the grouping of no tokens writes none
    ws = torch.empty(M.moe_route_backward_workspace_size(0, 3, E, H), dtype=torch.uint8, device=DEV)
    M.moe_route_backward(w, w.clone(), inv, xb, torch.ones((E, H), dtype=BF16, device=DEV), garbage,
                         torch.empty(0, dtype=torch.int32, device=DEV), w.clone(), e(0, H), dwr, db, ws)
    assert bool((dwr == 0).all()) and bool((db == 0).all())


def test_bad_slots_are_flagged_and_left_out():
    g = gen(3)
    T, H, k, R = 4, 72, 3, 12
    inv = routes(g, T, k)
    bad = inv.clone()
    bad[1, 1], bad[2, 0] = R, -2
    clean = torch.where((bad < 0) | (bad >= R), torch.full_like(bad, -1), bad)
    x, y = rand(g, T, H, F32), rand(g, R, H, F32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, out2 = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    M.moe_collect(y, bad, None, out, dev_status=status)
    M.moe_collect(y, clean, None, out2)
    assert int(status) == _lib.MOE_DEV_BAD_EXPERT and torch.equal(out, out2)
    status.zero_()
    xp, xp2 = torch.zeros((R, H), device=DEV), torch.zeros((R, H), device=DEV)
    M.moe_dispatch(x, bad, xp, dev_status=status)
    M.moe_dispatch(x, clean, xp2)
    assert int(status) == _lib.MOE_DEV_BAD_EXPERT and torch.equal(xp, xp2)
    M.moe_dispatch(x, bad, xp)  # without a status word


def test_special_values_follow_the_formula():
    inf = float("inf")
    y = torch.tensor([[1.0, inf, NAN, -inf], [2.0, 3.0, 1.0, inf]], device=DEV)
    inv = torch.tensor([[0, 1], [1, -1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1.0, 1.0], [0.0, 5.0]], device=DEV)
    # one slot may be read twice by a sum
    out = torch.empty((2, 4), device=DEV)
    M.moe_collect(y, inv, w, out)
    want = torch.tensor([[3.0, inf, NAN, NAN], [0.0, 0.0, 0.0, NAN]], device=DEV)
    assert torch.equal(torch.nan_to_num(out, 9e9, 8e8, -8e8), torch.nan_to_num(want, 9e9, 8e8, -8e8))


def test_rows_beyond_32_bit_offsets():
    """A row stride that puts the last slots past 2^31 elements."""
    T, k, H, ld = 70, 32, 64, 1 << 20
    R = T * k
    buf = torch.empty(((R - 1) * ld + H,), dtype=BF16, device=DEV)
    rows = torch.as_strided(buf, (R, H), (ld, 1))
    assert (R - 1) * ld > 2 ** 31
    g = gen(11)
    inv = routes(g, T, k)
    x, w = rand(g, T, H, BF16), torch.rand((T, k), generator=g, device=DEV)
    rows.zero_()
    M.moe_dispatch(x, inv, rows, w=w)
    near(rows, ref.spread(x, inv, w, torch.zeros((R, H), dtype=BF16, device=DEV)))
    out, dw = torch.empty((T, H), device=DEV), torch.empty((T, k), device=DEV)
    M.moe_dispatch_backward(rows, inv, out, w=w, x=x, dw=dw)
    near(out, ref.join(rows, inv, w, None, F32))
    near(dw, ref.dots(rows, inv, x))


# -- block norm --------------------------------------------------------------
GATES = ["none", "channel", "token", "full"]


def make_gate(kind, g, T, H, y_type, pad=0, shift=0):
    if kind == "none":
        return None
    if kind == "channel":
        return torch.randn(H, generator=g, device=DEV)
    if kind == "token":
        return torch.randn((T, 1), generator=g, device=DEV)
    return rand(g, T, H, y_type, pad, shift)


def norm_case(T, H, types, gate_kind, post, pad, shift, seed, scale=0.75, eps=1e-6, gammas=True):
    xt, yt = types
    g = gen(seed)
    x, y = rand(g, T, H, xt, pad, shift, 2.0), rand(g, T, H, yt, pad, shift, 0.5)
    gate = make_gate(gate_kind, g, T, H, yt, pad, shift)
    gp = 0.2 * torch.randn(H, generator=g, device=DEV) if gammas and post else None
    gq = 0.2 * torch.randn(H, generator=g, device=DEV) if gammas else None
    xo, xbuf = view(T, H, xt, pad, shift)
    n, nbuf = view(T, H, yt, pad, shift)
    r1 = torch.full((T,), NAN, device=DEV) if post else None
    r2 = torch.full((T,), NAN, device=DEV)
    M.moe_block_norm(x, y, xo, n, gamma_post=gp, gamma_pre=gq, gate=gate, scale=scale, eps=eps, post_norm=post,
                     rstd_post=r1, rstd_pre=r2)
    want = ref.norm(x, y, gate, gp, gq, scale, eps, post, xt, yt)
    near(xo, want["x_out"], "x_out")
    near(n, want["n_out"], "n_out")
    near(r2, want["rstd_pre"], "rstd_pre")
    if post:
        near(r1, want["rstd_post"], "rstd_post")
    untouched(xbuf, xo)
    untouched(nbuf, n)

    dxo, dn = rand(g, T, H, xt, pad, shift), rand(g, T, H, yt, pad, shift)
    dx, dxbuf = view(T, H, xt, pad, shift)
    dy, dybuf = view(T, H, yt, pad, shift)
    if gate is None:
        dgate, gbuf = None, None
    elif gate_kind == "full":
        dgate, gbuf = view(T, H, yt, pad, shift)
    else:
        dgate, gbuf = torch.full_like(gate, NAN), None
    dgp = torch.full((H,), NAN, device=DEV) if post else None
    dgq = torch.full((H,), NAN, device=DEV)
    ws = torch.empty(M.moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    M.moe_block_norm_backward(dxo, dn, xo, y, dx, dy, ws, gamma_post=gp, gamma_pre=gq, gate=gate, scale=scale,
                              post_norm=post, rstd_post=r1, rstd_pre=r2, dgate=dgate, dgamma_post=dgp, dgamma_pre=dgq)
    want = ref.norm_grad(dxo, dn, xo, y, gate, gp, gq, scale, r1, r2, post, xt, yt)
    for name, got in (("dx", dx), ("dy", dy), ("dgate", dgate), ("dgamma_post", dgp), ("dgamma_pre", dgq)):
        if got is not None:
            near(got, want[name], name)
    untouched(dxbuf, dx)
    untouched(dybuf, dy)
    if gbuf is not None:
        untouched(gbuf, dgate)


NORM_SIZES = [(1, 1), (1, 2560), (3, 8), (2, 31), (5, 257), (7, 520), (16, 2560), (33, 1001), (3, 4096), (3, 4104),
              (2, 8192), (2, 8200), (3, 16384), (1, 16383), (1300, 256), (2500, 64), (701, 640), (450, 2560),
              (317, 4200), (309, 9000), (160, 8191)]


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1), (2, 2)])
def test_block_norm_sizes(T, H, types, pad, shift):
    norm_case(T, H, (types[1], types[0]), "channel", True, pad, shift, seed=T * 131 + H)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("T,H", [(40, 264), (40, 333), (6, 5000), (5, 9000), (160, 8192)])
def test_block_norm_gates(gate, post, types, T, H):
    norm_case(T, H, (types[1], types[0]), gate, post, 0, 0, seed=T + H, scale=1.0, gammas=H % 2 == 0)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_block_norm_width_one(gate, types):
    """A [T, 1] gate is the full one where its type is y's."""
    norm_case(20, 1, types, gate, True, 3, 1, seed=4)


def test_block_norm_small_rows_with_eps_zero():
    """Rows of 1e-15 with eps = 0: factors of 1e15, whose cube fp32 cannot hold."""
    g = gen(2)
    T, H = 4, 256
    x, y = rand(g, T, H, F32, std=1e-15), rand(g, T, H, F32, std=1e-15)
    xo, n = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    r1, r2 = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    M.moe_block_norm(x, y, xo, n, gate=torch.full((H,), 1e-15, device=DEV), eps=0.0, rstd_post=r1, rstd_pre=r2)
    gate = torch.full((H,), 1e-15, device=DEV)
    dxo, dn = rand(g, T, H, F32), rand(g, T, H, F32)
    dx, dy, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gate)
    ws = torch.empty(M.moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    M.moe_block_norm_backward(dxo, dn, xo, y, dx, dy, ws, gate=gate, rstd_post=r1, rstd_pre=r2, dgate=dg)
    want = ref.norm_grad(dxo, dn, xo, y, gate, None, None, 1.0, r1, r2, True, F32, F32)
    for name, got in (("dx", dx), ("dy", dy), ("dgate", dg)):
        near(got, want[name], name)


@pytest.mark.parametrize("T,H", [(40, 257), (37, 2560), (7, 5001)])
@pytest.mark.parametrize("gate", ["token", "full"])
def test_block_norm_rows_on_odd_elements(T, H, gate):
    """bf16 rows whose starts alternate between the halves of a word, beside NaN in the gaps."""
    norm_case(T, H, (BF16, BF16), gate, True, 1 + H % 2, 1, seed=T)
    g = gen(T)
    x, y = rand(g, T, H, BF16), rand(g, T, H, BF16)
    xg = torch.full((T, H + 1 + H % 2), NAN, dtype=BF16, device=DEV)
    yg = xg.clone()
    xg[:, :H], yg[:, :H] = x, y
    outs = [torch.empty((T, H), dtype=BF16, device=DEV) for _ in range(4)]
    M.moe_block_norm(x, y, outs[0], outs[1])
    M.moe_block_norm(xg[:, :H], yg[:, :H], outs[2], outs[3])
    near(outs[2], ref.norm(x, y, None, None, None, 1.0, 1e-6, True, BF16, BF16)["x_out"])
    near(outs[3], ref.norm(x, y, None, None, None, 1.0, 1e-6, True, BF16, BF16)["n_out"])


def test_block_norm_zero_row_and_special_rows():
    """A row of zeros has factor 1/sqrt(eps); a NaN or an infinity stays in its own row."""
    x = torch.zeros((4, 40), device=DEV)
    y = torch.ones((4, 40), device=DEV)
    y[0] = 0
    y[1, 3], y[2, 5] = NAN, float("inf")
    xo, n, r2 = torch.empty_like(x), torch.empty_like(x), torch.empty(4, device=DEV)
    M.moe_block_norm(x, y, xo, n, eps=1e-4, rstd_pre=r2)
    assert bool((xo[0] == 0).all()) and bool((n[0] == 0).all()) and abs(float(r2[0]) - 100.0) < 1e-4
    assert bool(torch.isnan(n[1]).all()) and bool(torch.isnan(n[2]).all())
    assert bool(torch.isfinite(n[3]).all())


@pytest.mark.parametrize("types", TYPES, ids=str)
def test_block_norm_parts(types):
    """No block before, no norm after, no direct gradient, gradients not wanted, in place."""
    xt, yt = types[1], types[0]
    g = gen(21)
    T, H, scale, eps = 19, 328, 0.5, 1e-5
    x, y = rand(g, T, H, xt), rand(g, T, H, yt)
    gq = 0.2 * torch.randn(H, generator=g, device=DEV)
    r1, r2 = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    n, xo = torch.empty((T, H), dtype=yt, device=DEV), torch.empty((T, H), dtype=xt, device=DEV)
    # the norm alone
    M.moe_block_norm(x, None, None, n, gamma_pre=gq, eps=eps, rstd_pre=r2)
    want = ref.norm(x, None, None, None, gq, 1.0, eps, False, xt, yt)
    near(n, want["n_out"])
    near(r2, want["rstd_pre"])
    dn, dxo = rand(g, T, H, yt), rand(g, T, H, xt)
    dx, dgq = torch.empty_like(x), torch.empty(H, device=DEV)
    ws = torch.empty(M.moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    M.moe_block_norm_backward(None, dn, x, None, dx, None, ws, gamma_pre=gq, rstd_pre=r2, dgamma_pre=dgq)
    want = ref.norm_grad(None, dn, x, None, None, None, gq, 1.0, None, r2, False, xt, yt)
    near(dx, want["dx"])
    near(dgq, want["dgamma_pre"])
    # no norm after it, in place
    wantf = ref.norm(x, y, None, None, None, scale, eps, True, xt, yt)
    xin = x.clone()
    M.moe_block_norm(xin, y, xin, None, scale=scale, eps=eps, rstd_post=r1)
    near(xin, wantf["x_out"])
    dy = torch.empty_like(y)
    dxin = dxo.clone()
    want = ref.norm_grad(dxo, None, None, y, None, None, None, scale, r1, None, True, xt, yt)
    M.moe_block_norm_backward(dxin, None, None, y, dxin, dy, None, scale=scale, rstd_post=r1)
    near(dxin, want["dx"])
    near(dy, want["dy"])


def test_block_norm_bits_repeat_and_do_not_depend_on_the_workspace():
    g = gen(1)
    T, H = 3000, 2560
    x, y, dxo, dn = (rand(g, T, H, F32) for _ in range(4))
    gate = torch.randn(H, generator=g, device=DEV)
    r1, r2 = torch.rand(T, device=DEV), torch.rand(T, device=DEV)
    got = []
    for fill in (0, 255):
        ws = torch.full((M.moe_block_norm_workspace_size(T, H),), fill, dtype=torch.uint8, device=DEV)
        outs = [torch.empty_like(x), torch.empty_like(x)] + [torch.empty(H, device=DEV) for _ in range(3)]
        M.moe_block_norm_backward(dxo, dn, x, y, outs[0], outs[1], ws, gate=gate, rstd_post=r1, rstd_pre=r2,
                                  dgate=outs[2], dgamma_post=outs[3], dgamma_pre=outs[4])
        got.append(outs)
    assert all(torch.equal(a, b) for a, b in zip(*got))


# -- router gradient ---------------------------------------------------------
def group(ids, E):
    T, k = ids.shape
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, offsets, perm, inv = (torch.empty(n, **i32) for n in (E, E + 1, T * k, T * k))
    status = torch.zeros(1, **i32)
    _lib.moe_permute(ids, E, None, counts, offsets, perm, inv, None, status)
    assert int(status) == 0
    return offsets, perm


def route_case(T, H, k, E, dtype, pad, shift, seed, hot=None, same=False):
    g = gen(seed)
    score = torch.rand((T, E), generator=g, device=DEV)
    if hot is not None:
        score[:, :hot] += 1.0  # every token takes the first experts
    top, ids = score.topk(k, dim=1)
    ids = ids.to(torch.int32).contiguous()
    if same:
        ids.fill_(E - 1)  # the same expert k times
    w = torch.softmax(3 * top, dim=1).contiguous()
    x, wr = rand(g, T, H, BF16, pad, shift), rand(g, E, H, BF16, pad, shift, 0.02)
    dw, add = torch.randn((T, k), generator=g, device=DEV), rand(g, T, H, dtype, pad, shift)
    offsets, perm = group(ids, E)
    dl = torch.full((T, k), NAN, device=DEV)
    dx, dxbuf = view(T, H, dtype, pad, shift)
    dwr, dwbuf = view(E, H, F32, pad, shift)
    db = torch.full((E,), NAN, device=DEV)
    n = M.moe_route_backward_workspace_size(T, k, E, H)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, dl, dx, dwr, db, ws[:n], add=add, dev_status=status)
    want = ref.route_grad(dw, w, ids, x, wr, add, dtype)
    for name, got in (("dlogits", dl), ("dx", dx), ("dw_router", dwr), ("dbias", db)):
        near(got, want[name], name)
    assert int(status) == 0 and bool((ws[n:] == 255).all())
    untouched(dxbuf, dx)
    untouched(dwbuf, dwr)


@pytest.mark.parametrize("T,H,k,E,hot", [
    (1, 1, 1, 1, None), (1, 256, 4, 64, None), (16, 2560, 10, 512, None), (16, 256, 4, 64, None),
    (37, 1001, 3, 5, None), (300, 128, 8, 8, None), (1000, 2560, 10, 512, None), (1025, 136, 32, 1024, 40),
    (2100, 72, 2, 9, 2), (777, 4100, 5, 33, 5), (256, 64, 1, 3, 1), (257, 64, 1, 3, 1), (2, 65536, 2, 4, None),
])
@pytest.mark.parametrize("dtype,pad,shift", [(F32, 0, 0), (BF16, 8, 0), (F32, 3, 1), (BF16, 2, 2)], ids=str)
def test_route_gradient(T, H, k, E, hot, dtype, pad, shift):
    route_case(T, H, k, E, dtype, pad, shift, seed=T + H + k + E, hot=hot)


def test_route_gradient_through_column_slabs():
    """Enough routed elements for dx to read the router from shared memory: a ragged last slab, one and several
    chunks of routes per token, more experts than fit, and an ID out of range."""
    for T, H, k, E, dtype in ((6000, 1000, 9, 77, F32), (2100, 1544, 17, 64, BF16), (6000, 1000, 9, 1000, F32)):
        assert T * H * k >= 50_000_000
        route_case(T, H, k, E, dtype, 0, 0, seed=T)
    T, H, k, E = 6000, 1000, 9, 77
    g = gen(5)
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)[1].to(torch.int32).contiguous()
    bad = ids.clone()
    bad[17, 3], bad[5999, 8] = E, -1
    w = dw = torch.rand((T, k), generator=g, device=DEV)
    x, wr, status = rand(g, T, H, BF16), rand(g, E, H, BF16), torch.zeros(1, dtype=torch.int32, device=DEV)
    offsets, perm = group(ids, E)
    dl, dx = torch.empty((T, k), device=DEV), torch.empty((T, H), device=DEV)
    M.moe_route_backward(dw, w, bad, x, wr, offsets, perm, dl, dx, None, None, None, dev_status=status)
    assert int(status) == _lib.MOE_DEV_BAD_EXPERT
    near(dx, ref.join(wr, torch.where(bad == E, torch.full_like(bad, -1), bad), dl, None, F32))


def test_route_gradient_same_expert_in_every_place():
    route_case(200, 96, 6, 7, F32, 0, 0, seed=3, same=True)


def test_route_gradient_parts_and_bits():
    g = gen(31)
    T, H, k, E = 700, 320, 4, 6
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)[1].to(torch.int32).contiguous()
    w = torch.softmax(torch.randn((T, k), generator=g, device=DEV), 1)
    dw = torch.randn((T, k), generator=g, device=DEV)
    x, wr = rand(g, T, H, BF16), rand(g, E, H, BF16)
    offsets, perm = group(ids, E)
    ws = torch.empty(M.moe_route_backward_workspace_size(T, k, E, H), dtype=torch.uint8, device=DEV)
    new = lambda: (torch.empty((T, k), device=DEV), torch.empty((T, H), device=DEV), torch.empty((E, H), device=DEV),
                   torch.empty(E, device=DEV))
    a, b = new(), new()
    for dl, dx, dwr, db in (a, b):
        M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, dl, dx, dwr, db, ws)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    c = new()
    M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, c[0], c[1], None, None, None)
    M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, c[0], None, c[2], None, ws)
    M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, c[0], None, None, c[3], ws)
    assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_route_gradient_bad_grouping_is_flagged():
    g = gen(32)
    T, H, k, E = 20, 64, 2, 4
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)[1].to(torch.int32).contiguous()
    w = dw = torch.rand((T, k), generator=g, device=DEV)
    x, wr = rand(g, T, H, BF16), rand(g, E, H, BF16)
    offsets, perm = group(ids, E)
    ws = torch.empty(M.moe_route_backward_workspace_size(T, k, E, H), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dl, dwr, db = torch.empty((T, k), device=DEV), torch.full((E, H), 5.0, device=DEV), torch.full((E,), 5.0, device=DEV)
    for i, v in ((0, 1), (2, 1 << 30), (1, -5), (E, 0)):
        bad = offsets.clone()
        bad[i] = v
        status.zero_()
        M.moe_route_backward(dw, w, ids, x, wr, bad, perm, dl, None, dwr, db, ws, dev_status=status)
        assert int(status) == _lib.MOE_DEV_BAD_EXPERT
        assert bool((dwr == 5).all()) and bool((db == 5).all())
    bad = perm.clone()
    bad[3], bad[7] = T * k, -1
    status.zero_()
    M.moe_route_backward(dw, w, ids, x, wr, offsets, bad, dl, None, dwr, db, ws, dev_status=status)
    assert int(status) == _lib.MOE_DEV_BAD_EXPERT and bool((dwr != 5).all())
    for v in (E, -1, -3):
        bad = ids.clone()
        bad[4, 1] = v
        status.zero_()
        dx = torch.empty((T, H), device=DEV)
        M.moe_route_backward(dw, w, bad, x, wr, offsets, perm, dl, dx, None, None, None, dev_status=status)
        assert int(status) == _lib.MOE_DEV_BAD_EXPERT
        one = torch.tensor([[int(ids[4, 0]), -1]], dtype=torch.int32, device=DEV)  # the other route is left out
        near(dx[4:5], ref.join(wr, one, dl[4:5], None, F32))


# -- how calls are made ------------------------------------------------------
def test_refusals_of_the_binding():
    x, inv = torch.zeros((4, 64), device=DEV), torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    xp = torch.zeros((8, 64), device=DEV)

    def refused(status, f, *a, **kw):
        with pytest.raises(MoEError) as e:
            f(*a, **kw)
        assert e.value.status == status, e.value

    refused(_lib.MOE_EINVAL, M.moe_dispatch, x.half(), inv, xp)
    refused(_lib.MOE_EINVAL, M.moe_dispatch, x, inv, xp.to(BF16))
    refused(_lib.MOE_EINVAL, M.moe_dispatch, x, inv.long(), xp)
    refused(_lib.MOE_EINVAL, M.moe_dispatch, x, inv.cpu(), xp)
    refused(_lib.MOE_EINVAL, M.moe_dispatch, x.t().contiguous().t(), inv, xp)
    refused(_lib.MOE_ESHAPE, M.moe_dispatch, x, inv[:3], xp)
    refused(_lib.MOE_ESHAPE, M.moe_dispatch, x, inv, xp[:, :60])
    refused(_lib.MOE_ESHAPE, M.moe_dispatch, x, inv, xp[:1].expand(8, 64))
    # more rows than the C ABI's int holds (one row in memory, seen 2^32 + 8 times)
    refused(_lib.MOE_ENOTSUP, M.moe_dispatch, x, inv, xp[:1].expand((1 << 32) + 8, 64))
    refused(_lib.MOE_ESHAPE, M.moe_dispatch, x, inv, xp, w=torch.zeros((4, 3), device=DEV))
    refused(_lib.MOE_EINVAL, M.moe_dispatch, x, inv, xp, w=torch.zeros((2, 4), device=DEV).t())
    refused(_lib.MOE_EINVAL, M.moe_dispatch_backward, xp, inv, x, dw=torch.zeros((4, 2), device=DEV))
    refused(_lib.MOE_EINVAL, M.moe_block_norm, x, None, x, None)
    refused(_lib.MOE_ESHAPE, M.moe_block_norm, x, x.clone(), x, x.clone(), gate=torch.zeros(63, device=DEV))
    refused(_lib.MOE_EINVAL, M.moe_block_norm, x, x.clone(), x, x.clone(), gate=torch.zeros(64, device=DEV, dtype=BF16))
    refused(_lib.MOE_EINVAL, M.moe_block_norm, x, x.clone(), x, x.clone(), gamma_post=torch.zeros(64, device=DEV),
            post_norm=False)
    assert bool((xp == 0).all())


def _block_step(s):
    """dispatch -> collect -> norms -> their gradients -> router gradient, all into s's buffers."""
    M.moe_dispatch(s["x"], s["inv"], s["xp"])
    M.moe_collect(s["xp"], s["inv"], s["w"], s["y"])
    M.moe_block_norm(s["res"], s["y"], s["xo"], s["n"], gate=s["gate"], rstd_post=s["r1"], rstd_pre=s["r2"])
    M.moe_block_norm_backward(s["dres"], s["dn"], s["xo"], s["y"], s["dx"], s["dy"], s["ws"], gate=s["gate"],
                              rstd_post=s["r1"], rstd_pre=s["r2"], dgate=s["dgate"], dgamma_post=s["dgp"],
                              dgamma_pre=s["dgq"])
    M.moe_collect_backward(s["dy"], s["xp"], s["inv"], s["w"], s["dxp"], s["dw"])
    M.moe_dispatch_backward(s["dxp"], s["inv"], s["dtok"])
    M.moe_route_backward(s["dw"], s["w"], s["ids"], s["x"], s["wr"], s["offsets"], s["perm"], s["dl"], s["dtok"],
                         s["dwr"], s["db"], s["ws2"], add=s["dtok"])
    return [s[k] for k in ("xo", "n", "dx", "dy", "dgate", "dgp", "dgq", "dxp", "dw", "dtok", "dl", "dwr", "db")]


def _block_state(seed, T=96, H=512, k=4, E=16):
    g = gen(seed)
    s = {"x": rand(g, T, H, BF16), "wr": rand(g, E, H, BF16, std=0.02), "res": rand(g, T, H, F32),
         "dres": rand(g, T, H, F32), "dn": rand(g, T, H, BF16), "gate": torch.randn(H, generator=g, device=DEV)}
    top, ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)
    s["ids"], s["w"] = ids.to(torch.int32).contiguous(), torch.softmax(top, 1)
    s["offsets"], s["perm"] = group(s["ids"], E)
    s["inv"] = torch.empty((T * k,), dtype=torch.int32, device=DEV)
    s["inv"][s["perm"].long()] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    s["inv"] = s["inv"].view(T, k)
    e = lambda *sh, t=F32: torch.zeros(sh, dtype=t, device=DEV)
    s.update(xp=e(T * k, H, t=BF16), dxp=e(T * k, H, t=BF16), y=e(T, H, t=BF16), xo=e(T, H), n=e(T, H, t=BF16),
             r1=e(T), r2=e(T), dx=e(T, H), dy=e(T, H, t=BF16), dgate=e(H), dgp=e(H), dgq=e(H), dw=e(T, k),
             dtok=e(T, H), dl=e(T, k), dwr=e(E, H), db=e(E))
    s["ws"] = torch.empty(M.moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    s["ws2"] = torch.empty(M.moe_route_backward_workspace_size(T, k, E, H), dtype=torch.uint8, device=DEV)
    return s


def test_captured_replayed_and_on_another_stream():
    s = _block_state(1)
    want = [t.clone() for t in _block_step(s)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for t in _block_step(s):
            t.zero_()
        got = [t.clone() for t in _block_step(s)]
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _block_step(s)
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    # other inputs in the same buffers
    other = _block_state(2)
    want = [t.clone() for t in _block_step(other)]
    for k in ("x", "wr", "res", "dres", "dn", "gate", "ids", "w", "offsets", "perm", "inv"):
        s[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_explicit_stream_and_two_calls_at_once():
    a, b = _block_state(3), _block_state(4)
    wa, wb = ([t.clone() for t in _block_step(s)] for s in (a, b))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s in ((s1, a), (s2, b)):
            with torch.cuda.stream(st):
                outs = _block_step(s)
    torch.cuda.synchronize()
    for s, w in ((a, wa), (b, wb)):
        assert all(torch.equal(p, q) for p, q in zip(w, _block_step(s)))
    a["xp"].zero_()
    torch.cuda.synchronize()
    M.moe_dispatch(a["x"], a["inv"], a["xp"], stream=s1)
    s1.synchronize()
    near(a["xp"], ref.spread(a["x"], a["inv"], None, torch.zeros_like(a["xp"])))


@pytest.mark.parametrize("gates", ["none", "channel", "token"])
def test_stack_with_norms_after_the_layers(gates):
    """MoEStack with post norms: each layer's output as MoELayer gives it, then
    the definition of the norms, rounded to the stream's and the router's types
    at the same places."""
    import workloads as wl

    cfg, L, T, eps, scale = wl.TINY, 3, 16, 1e-6, 0.5
    g = gen(91)
    H = cfg.H
    data = [wl.layer_inputs(cfg, DEV, layer=l) for l in range(L)]
    vec = lambda: [0.2 * torch.randn(H, generator=g, device=DEV) for _ in range(L)]
    gammas, post = vec(), vec()
    gate = {"none": None, "channel": [1 + v for v in vec()],
            "token": [torch.rand((T, 1), generator=g, device=DEV) for _ in range(L)]}[gates]
    layers = [M.MoELayer(d["w_router"], d["bias"], d["w_gateup"], d["w_down"], cfg.k, T) for d in data]
    x0 = torch.randn((T, H), generator=g, device=DEV)
    stack = M.MoEStack(layers, T, eps, gammas, post_gammas=post, gates=gate, scale=scale)
    x = stack.forward(x0.clone())
    # the same layers, one call at a time
    want, n = x0.clone(), torch.empty((T, H), dtype=BF16, device=DEV)
    _lib.moe_rmsnorm(want, gammas[0], eps, n)
    for l in range(L):
        y = layers[l].forward(n).clone()
        ref_l = ref.norm(want, y, None if gate is None else gate[l], post[l], gammas[l + 1] if l + 1 < L else None,
                         scale, eps, True, F32, BF16)
        nxt = torch.empty_like(want)
        M.moe_block_norm(want, y, nxt, n, gamma_post=post[l], gamma_pre=gammas[l + 1] if l + 1 < L else None,
                         gate=None if gate is None else gate[l], scale=scale, eps=eps)
        near(nxt, ref_l["x_out"], f"layer {l}")
        near(n, ref_l["n_out"], f"layer {l}")
        want = nxt
    assert torch.equal(x, want)
    # standing alone, a layer makes its own norms
    y1 = x0.clone()
    for l in range(L):
        for call in stack.layer_calls(y1, l):
            M.MoELayer.issue(call)
    assert float((y1 - x).abs().max()) <= 2 ** -6 * float(x.abs().max())  # another bf16 rounding of n per layer
    assert all(m.read_status() == 0 for m in layers)


def test_a_block_forward_and_backward_against_autograd():
    """norm -> router -> dispatch -> one linear map per expert -> collect -> norms, and its gradients, chained as
    a training step chains them, against torch.autograd of the definition in 64 bits.

    fp32 rows, so the only bf16 roundings are those of the router's inputs, which both sides share.  Each value
    passes about 40 fp32 roundings on sums of up to H = 128 terms: (128 + 40) 2^-24 = 1e-5 of the terms' size
    per stage; five stages and cancellation within a factor 10 give 5e-4 of an output's largest value.
    """
    g = gen(77)
    T, H, k, E, eps, scale = 50, 128, 3, 8, 1e-5, 0.9
    x0 = rand(g, T, H, F32)
    we = torch.randn((E, H, H), generator=g, device=DEV) / H ** 0.5
    wr, bias = rand(g, E, H, BF16, std=0.3), torch.randn(E, generator=g, device=DEV)
    gq, gp, gq2 = (0.1 * torch.randn(H, generator=g, device=DEV) for _ in range(3))
    gate = torch.rand(H, generator=g, device=DEV)
    a, b = rand(g, T, H, F32), rand(g, T, H, F32)  # gradients of the block's two outputs
    f = lambda *s: torch.empty(s, device=DEV)

    # forward
    n, r0 = f(T, H), f(T)
    M.moe_block_norm(x0, None, None, n, gamma_pre=gq, eps=eps, rstd_pre=r0)
    nb = n.to(BF16)
    ids, w, gap = torch.empty((T, k), dtype=torch.int32, device=DEV), f(T, k), f(T)
    _lib.moe_route(nb, wr, bias, k, ids, w, gap,
                   torch.empty(_lib.route_workspace_size(T, E), dtype=torch.uint8, device=DEV))
    offsets, perm = group(ids, E)
    inv = torch.empty(T * k, dtype=torch.int32, device=DEV)
    inv[perm.long()] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    inv = inv.view(T, k)
    xp, y, xo, n2, r1, r2 = f(T * k, H), f(T, H), f(T, H), f(T, H), f(T), f(T)
    M.moe_dispatch(n, inv, xp)
    owner = ids.view(-1)[perm.long()].long()
    yp = torch.einsum("rh,rhg->rg", xp, we[owner])
    M.moe_collect(yp, inv, w, y)
    M.moe_block_norm(x0, y, xo, n2, gamma_post=gp, gamma_pre=gq2, gate=gate, scale=scale, eps=eps, rstd_post=r1,
                     rstd_pre=r2)
    # backward
    dx, dy, dgate, dgp, dgq2, dgq = f(T, H), f(T, H), f(H), f(H), f(H), f(H)
    ws = torch.empty(M.moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    M.moe_block_norm_backward(a, b, xo, y, dx, dy, ws, gamma_post=gp, gamma_pre=gq2, gate=gate, scale=scale,
                              rstd_post=r1, rstd_pre=r2, dgate=dgate, dgamma_post=dgp, dgamma_pre=dgq2)
    dyp, dw = f(T * k, H), f(T, k)
    M.moe_collect_backward(dy, yp, inv, w, dyp, dw)
    dxp = torch.einsum("rg,rhg->rh", dyp, we[owner])
    dn = f(T, H)
    M.moe_dispatch_backward(dxp, inv, dn)
    dl, dwr, db = f(T, k), f(E, H), f(E)
    ws2 = torch.empty(M.moe_route_backward_workspace_size(T, k, E, H), dtype=torch.uint8, device=DEV)
    M.moe_route_backward(dw, w, ids, nb, wr, offsets, perm, dl, dn, dwr, db, ws2, add=dn)
    dx0 = f(T, H)
    # the stream's direct gradient joins after the first norm's (its x_out is x0 itself)
    M.moe_block_norm_backward(dx, dn, x0, None, dx0, None, ws, gamma_pre=gq, rstd_pre=r0, dgamma_pre=dgq)

    # the definition
    leaf = lambda t: t.to(torch.float64).requires_grad_()
    X, WR, B, GQ, GP, GQ2, G = map(leaf, (x0, wr, bias, gq, gp, gq2, gate))
    rms = lambda v: v / (v.square().mean(-1, keepdim=True) + eps).sqrt()
    N = rms(X) * (1 + GQ)
    NB = nb.to(torch.float64) + (N - N.detach())  # the router reads the rounded rows; rounding passes gradients on
    W = torch.softmax((NB @ WR.t() + B).gather(1, ids.long()), 1)
    V = torch.einsum("th,tkhg->tkg", N, we.to(torch.float64)[ids.long()])
    Y = (W[..., None] * V).sum(1)
    XO = scale * X + G * rms(Y) * (1 + GP)
    N2 = rms(XO) * (1 + GQ2)
    loss = (XO * a).sum() + (N2 * b).sum()
    loss.backward()
    for name, got, want in (("x_out", xo, XO), ("n_out", n2, N2), ("x", dx0, X.grad), ("w_router", dwr, WR.grad),
                            ("bias", db, B.grad), ("gamma_pre", dgq, GQ.grad), ("gamma_post", dgp, GP.grad),
                            ("gamma_pre of the next", dgq2, GQ2.grad), ("gate", dgate, G.grad)):
        want = want.detach()
        off = float((got.to(torch.float64) - want).abs().max())
        assert off <= 5e-4 * float(want.abs().max()), (name, off, float(want.abs().max()))
