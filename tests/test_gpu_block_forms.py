"""MoEStack's norms after the layers and the launch forms of libmoe_block that
only larger calls reach, against the definitions in 64 bits."""
import pytest
import torch

import block_reference as ref
import sparse_moe_routed_gb300 as M
import workloads as wl
from sparse_moe_routed_gb300 import _lib, pack_layer_experts
from test_gpu_block import group, near, rand, untouched, view

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def stack_of(L, T_max, g, **kw):
    H = wl.TINY.H
    data = [wl.layer_inputs(wl.TINY, DEV, layer=l) for l in range(L)]
    layers = [M.MoELayer(d["w_router"], d["bias"], d["w_gateup"], d["w_down"], wl.TINY.k, T_max) for d in data]
    vec = lambda: [0.2 * torch.randn(H, generator=g, device=DEV) for _ in range(L)]
    return M.MoEStack(layers, T_max, gammas=vec(), post_gammas=vec(), **kw)


def test_stack_follows_its_replaced_gates_and_scale():
    """The second forward on one stream buffer gives what a stack made with the new values gives."""
    g, L, T, T_max = gen(5), 2, 11, 16
    gates = lambda: [torch.rand((T_max, 1), generator=g, device=DEV) for _ in range(L)]
    s = stack_of(L, T_max, g, gates=gates(), scale=0.5)
    x0 = torch.randn((T, wl.TINY.H), generator=g, device=DEV)
    x = x0.clone()
    first = s.forward(x).clone()
    new = gates()
    for scale, eps in ((0.5, 1e-6), (0.75, 1e-2)):
        s.gates[:], s.scale, s.eps = new, scale, eps
        x.copy_(x0)
        got = s.forward(x).clone()
        fresh = M.MoEStack(s.layers, T_max, eps, s.gammas, post_gammas=s.post_gammas, gates=new, scale=scale)
        assert torch.equal(got, fresh.forward(x0.clone())) and not torch.equal(got, first)
    with pytest.raises(AssertionError):
        s.forward(torch.zeros((T_max + 1, wl.TINY.H), device=DEV))


@pytest.mark.parametrize("T,k,E,H,n", [
    (520, 1, 8, 264, 65),       # eight experts of one unit and one route: the most partial rows there can be
    (1032, 1, 8, 72, 129),      # the last unit of an expert holds one route
    (20000, 1, 2, 136, None),   # far more units than experts
    (16640, 8, 8, 64, None),    # units of 256 routes, every token in every expert
])
def test_router_gradient_fills_its_workspace(T, k, E, H, n):
    g = gen(T + E)
    if n is None:
        ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)[1].to(torch.int32).contiguous()
    else:
        ids = (torch.arange(T, device=DEV) % E).to(torch.int32).view(T, 1)
        assert T == n * E
    w, dw = torch.rand((T, k), generator=g, device=DEV), torch.randn((T, k), generator=g, device=DEV)
    x, wr = rand(g, T, H, BF16), rand(g, E, H, BF16)
    offsets, perm = group(ids, E)
    size = M.moe_route_backward_workspace_size(T, k, E, H)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device=DEV)
    dl, dx = torch.empty((T, k), device=DEV), torch.empty((T, H), device=DEV)
    dwr, db = torch.empty((E, H), device=DEV), torch.empty(E, device=DEV)
    M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, dl, dx, dwr, db, ws[:size])
    want = ref.route_grad(dw, w, ids, x, wr, None, F32)
    for name, got in (("dlogits", dl), ("dx", dx), ("dw_router", dwr), ("dbias", db)):
        near(got, want[name], name)
    assert bool((ws[size:] == 255).all())


@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=str)
def test_norm_gradient_of_no_rows_is_zero_whatever_the_gate_holds(value):
    H = 40
    e = lambda *s: torch.empty(s, device=DEV)
    cols = [torch.full((H,), 7.0, device=DEV) for _ in range(3)]
    ws = torch.empty(M.moe_block_norm_workspace_size(0, H), dtype=torch.uint8, device=DEV)
    full = lambda: torch.full((H,), value, device=DEV)
    M.moe_block_norm_backward(e(0, H), e(0, H), e(0, H), e(0, H), e(0, H), e(0, H), ws, gate=full(), gamma_post=full(),
                              gamma_pre=full(), rstd_post=e(0), rstd_pre=e(0), dgate=cols[0], dgamma_post=cols[1],
                              dgamma_pre=cols[2])
    assert all(bool((c == 0).all()) for c in cols)


def test_int4_launches_right_after_a_block_call_read_what_it_wrote():
    """moe_dispatch rewrites x_perm between the row gather and the gate/up launch, moe_collect_backward rewrites h
    between that and the down launch: both int4 launches start early and read the rows only after these calls."""
    cfg = wl.LayerConfig("int4_between", T=16, H=1024, E=64, k=4, I=256, bias=None, seed=53)
    T, k, E, H, I, R, fmt = 16, cfg.k, cfg.E, cfg.H, cfg.I, 64, _lib.MOE_W_INT4_G64_TILED
    d = wl.layer_inputs(cfg, DEV)
    q_gu, s_gu = wl.quantize_int4_g64(d["w_gateup"])
    q_d, s_d = wl.quantize_int4_g64(d["w_down"])
    gu, dn = pack_layer_experts(q_gu, q_d, _lib.MOE_W_INT4_G64, E, H, I, s_gateup=s_gu, s_down=s_d)
    g = gen(53)
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)[1].to(torch.int32).contiguous()
    x, x2, th = rand(g, T, H, BF16), rand(g, T, H, BF16), rand(g, T, I, BF16)
    w = torch.rand((T, k), generator=g, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, offsets, perm, inv = (torch.empty(n, **i32) for n in (E, E + 1, R, R))
    st = torch.zeros(1, **i32)

    def steps(wait):
        xp, h = torch.zeros((R, H), dtype=BF16, device=DEV), torch.zeros((R, I), dtype=BF16, device=DEV)
        y, slots = torch.zeros((R, H), device=DEV), inv.view(T, k)
        torch.cuda.synchronize()
        for call in (lambda: _lib.moe_permute(ids, E, x, counts, offsets, perm, inv, xp, st),
                     lambda: M.moe_dispatch(x2, slots, xp, w=w, dev_status=st),
                     lambda: _lib.moe_expert_gateup(xp, offsets, E, H, I, gu, h, st, fmt=fmt)):
            call()
            wait()
        h_gate = h.clone()
        for call in (lambda: _lib.moe_expert_gateup(xp, offsets, E, H, I, gu, h, st, fmt=fmt),
                     lambda: M.moe_collect_backward(th, None, slots, w, h, dev_status=st),
                     lambda: _lib.moe_expert_down(h, offsets, E, H, I, dn, y, st, fmt=fmt)):
            call()
            wait()
        return xp, h_gate, h, y

    want = steps(torch.cuda.synchronize)
    assert int(st) == 0 and bool((want[3] != 0).any())
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, steps(lambda: None)))
    assert int(st) == 0


# -- the forms that large calls take -----------------------------------------
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def warp_per_token(H):
    """Tokens from which one warp owns a token where weights have gradients, with its last CTA ragged: 24 warps per SM
    are wanted, and where a row is one piece of 256 columns half as many tokens leave no second CTA per token."""
    return 24 * sms() // (2 if H <= 256 else 1) // 4 * 4 + 5


def slots(g, T, k, drop):
    """Slots for T k routes among a few more rows, some routes and some whole tokens without one."""
    R = T * k + 5
    inv = torch.randperm(R, generator=g, device=DEV)[:T * k].to(torch.int32).view(T, k)
    if drop:
        gone = torch.rand((T, k), generator=g, device=DEV) < drop
        gone[T - 3:] = True
        inv = torch.where(gone, torch.full_like(inv, -1), inv)
    return R, inv.contiguous()


def check_chunks(T, near_rows, step=1024):
    """Compares a token range at a time: the reference holds [tokens, k, H] in 64 bits."""
    for a in range(0, T, step):
        near_rows(slice(a, min(T, a + step)))


@pytest.mark.parametrize("types", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)], ids=str)
@pytest.mark.parametrize("H,k,pad", [(264, 3, 0), (520, 10, 8), (1001, 17, 0), (136, 20, 0), (258, 32, 4), (513, 2, 1)])
def test_a_warp_per_token(H, k, pad, types):
    rows, tok = types
    T = warp_per_token(H)
    g = gen(H + k)
    R, inv = slots(g, T, k, 0.2)
    w = torch.randn((T, k), generator=g, device=DEV)
    used = torch.zeros(R, dtype=torch.bool, device=DEV)
    used[inv[inv >= 0].long()] = True
    yp = rand(g, R, H, rows, pad)
    yp[~used] = float("nan")
    x, dout, add = rand(g, T, H, rows, pad), rand(g, T, H, tok, pad), rand(g, T, H, tok, pad)
    dx, dw = torch.full((T, H + pad), 3.0, dtype=tok, device=DEV)[:, :H], torch.full((T, k), float("nan"), device=DEV)
    M.moe_dispatch_backward(yp, inv, dx, w=w, x=x, dw=dw, add=add)
    out = torch.full((T, H), 3.0, dtype=tok, device=DEV)
    M.moe_collect(yp, inv, w, out)
    dyp, dw2 = torch.full((R, H + pad), -7.0, dtype=rows, device=DEV)[:, :H], torch.full_like(dw, float("nan"))
    M.moe_collect_backward(dout, yp, inv, w, dyp, dw2)

    def rows_near(s):
        near(dx[s], ref.join(yp, inv[s], w[s], add[s], tok), "dx")
        near(out[s], ref.join(yp, inv[s], w[s], None, tok), "out")
        near(dw[s], ref.dots(yp, inv[s], x[s]), "dw of dispatch")
        near(dw2[s], ref.dots(yp, inv[s], dout[s]), "dw of collect")

    check_chunks(T, rows_near)
    near(dyp, ref.spread(dout, inv, w, torch.full_like(dyp, -7.0)), "dy_perm")


@pytest.mark.parametrize("rows", [F32, BF16], ids=str)
@pytest.mark.parametrize("H,k", [(64, 2), (72, 20), (264, 1), (131, 3)])
def test_a_warp_per_token_without_sums(H, k, rows):
    T = 120 * sms() + 1
    g = gen(T + H)
    R, inv = slots(g, T, k, 0.1)
    w, x = torch.randn((T, k), generator=g, device=DEV), rand(g, T, H, rows)
    for wt in (w, None):
        xp = torch.full((R, H), -7.0, dtype=rows, device=DEV)
        M.moe_dispatch(x, inv, xp, w=wt)
        near(xp, ref.spread(x, inv, wt, torch.full_like(xp, -7.0)), "x_perm")


@pytest.mark.parametrize("T,k,E,H,pad", [(13000, 8, 40, 264, 0), (12600, 8, 40, 136, 3), (33000, 4, 7, 72, 0)])
def test_router_gradient_in_units_of_256_routes(T, k, E, H, pad):
    assert T * k > 100_000
    g = gen(T)
    score = torch.rand((T, E), generator=g, device=DEV)
    score[:, :k] += 0.6  # a few experts of many units
    ids = score.topk(k, 1)[1].to(torch.int32).contiguous()
    w, dw = torch.rand((T, k), generator=g, device=DEV), torch.randn((T, k), generator=g, device=DEV)
    x, wr = rand(g, T, H, BF16, pad), rand(g, E, H, BF16, pad)
    offsets, perm = group(ids, E)
    ws = torch.empty(M.moe_route_backward_workspace_size(T, k, E, H), dtype=torch.uint8, device=DEV)
    dl, dx = torch.empty((T, k), device=DEV), torch.empty((T, H), device=DEV)
    dwr, db = torch.empty((E, H), device=DEV), torch.empty(E, device=DEV)
    M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, dl, dx, dwr, db, ws)
    want = ref.route_grad(dw, w, ids, x, wr, None, F32)
    for name, got in (("dlogits", dl), ("dx", dx), ("dw_router", dwr), ("dbias", db)):
        near(got, want[name], name)


# -- operands that differ in stride and alignment, offsets past 32 bits ------
LAYOUTS = [(0, 0), (8, 0), (3, 1), (2, 2), (1, 0), (16, 8), (5, 3), (0, 1)]  # pad, shift


def layout(i):
    return LAYOUTS[i % len(LAYOUTS)]


@pytest.mark.parametrize("turn", range(len(LAYOUTS)))
@pytest.mark.parametrize("T,H", [(37, 264), (9, 521), (5, 8300)])
@pytest.mark.parametrize("xt,yt", [(F32, BF16), (BF16, BF16), (BF16, F32)], ids=str)
def test_block_norm_operands_of_different_layouts(T, H, xt, yt, turn):
    g = gen(T + H + turn)
    new = lambda i, dtype: view(T, H, dtype, *layout(turn + i))
    x, y = rand(g, T, H, xt, *layout(turn)), rand(g, T, H, yt, *layout(turn + 1))
    gate = rand(g, T, H, yt, *layout(turn + 2))
    (xo, b0), (n, b1) = new(3, xt), new(4, yt)
    gp, gq = (0.2 * torch.randn(H, generator=g, device=DEV) for _ in range(2))
    r1, r2 = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    M.moe_block_norm(x, y, xo, n, gamma_post=gp, gamma_pre=gq, gate=gate, scale=0.75, rstd_post=r1, rstd_pre=r2)
    want = ref.norm(x, y, gate, gp, gq, 0.75, 1e-6, True, xt, yt)
    near(xo, want["x_out"], "x_out")
    near(n, want["n_out"], "n_out")
    dxo, dn = rand(g, T, H, xt, *layout(turn + 5)), rand(g, T, H, yt, *layout(turn + 6))
    (dx, b2), (dy, b3), (dg, b4) = new(7, xt), new(8, yt), new(10, yt)
    dgp, dgq = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    ws = torch.empty(M.moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    M.moe_block_norm_backward(dxo, dn, xo, y, dx, dy, ws, gamma_post=gp, gamma_pre=gq, gate=gate, scale=0.75,
                              rstd_post=r1, rstd_pre=r2, dgate=dg, dgamma_post=dgp, dgamma_pre=dgq)
    want = ref.norm_grad(dxo, dn, xo, y, gate, gp, gq, 0.75, r1, r2, True, xt, yt)
    for name, got in (("dx", dx), ("dy", dy), ("dgate", dg), ("dgamma_post", dgp), ("dgamma_pre", dgq)):
        near(got, want[name], name)
    for buf, v in ((b0, xo), (b1, n), (b2, dx), (b3, dy), (b4, dg)):
        untouched(buf, v)


@pytest.mark.parametrize("turn", range(len(LAYOUTS)))
@pytest.mark.parametrize("T,H,k", [(37, 264, 4), (300, 77, 3)])
@pytest.mark.parametrize("rows,tok", [(F32, BF16), (BF16, BF16), (BF16, F32)], ids=str)
def test_row_movements_and_router_gradient_of_different_layouts(T, H, k, rows, tok, turn):
    g = gen(T + H + turn)
    R, inv = slots(g, T, k, 0.1)
    w = torch.randn((T, k), generator=g, device=DEV)
    at = lambda i: layout(turn + i)
    x, yp, dout, add = (rand(g, n, H, t, *at(i)) for i, (n, t) in enumerate(((T, rows), (R, rows), (T, tok), (T, tok))))
    (dx, b0), (dyp, b1), (out, b2) = view(T, H, tok, *at(4)), view(R, H, rows, *at(5)), view(T, H, tok, *at(6))
    dw, dw2 = torch.empty((T, k), device=DEV), torch.empty((T, k), device=DEV)
    M.moe_dispatch_backward(yp, inv, dx, w=w, x=x, dw=dw, add=add)
    M.moe_collect(yp, inv, w, out, add=add)
    M.moe_collect_backward(dout, yp, inv, w, dyp, dw2)
    near(dx, ref.join(yp, inv, w, add, tok), "dx")
    near(out, ref.join(yp, inv, w, add, tok), "out")
    near(dw, ref.dots(yp, inv, x), "dw of dispatch")
    near(dw2, ref.dots(yp, inv, dout), "dw of collect")
    near(dyp, ref.spread(dout, inv, w, torch.full_like(dyp, -7.0)), "dy_perm")
    for buf, v in ((b0, dx), (b1, dyp), (b2, out)):
        untouched(buf, v)
    E = 6
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)[1].to(torch.int32).contiguous()
    offsets, perm = group(ids, E)
    xb, wr = rand(g, T, H, BF16, *at(1)), rand(g, E, H, BF16, *at(2))
    (dx, b0), (dwr, b1) = view(T, H, tok, *at(3)), view(E, H, F32, *at(4))
    dl, db = torch.empty((T, k), device=DEV), torch.empty(E, device=DEV)
    ws = torch.empty(M.moe_route_backward_workspace_size(T, k, E, H), dtype=torch.uint8, device=DEV)
    M.moe_route_backward(dw, w, ids, xb, wr, offsets, perm, dl, dx, dwr, db, ws, add=add)
    want = ref.route_grad(dw, w, ids, xb, wr, add, tok)
    for name, got in (("dlogits", dl), ("dx", dx), ("dw_router", dwr), ("dbias", db)):
        near(got, want[name], name)
    untouched(b0, dx)
    untouched(b1, dwr)


@pytest.mark.parametrize("H", [64, 63])
def test_norms_and_router_gradient_of_rows_past_32_bit_offsets(H):
    T, k, E, ld = 2100, 2, 5, 1 << 20
    assert (T - 1) * ld > 2 ** 31
    g = gen(H)
    far = lambda: torch.as_strided(torch.empty((T - 1) * ld + H, dtype=BF16, device=DEV), (T, H), (ld, 1))
    x, out = far(), far()
    x.copy_(torch.randn((T, H), generator=g, device=DEV))
    out.zero_()
    y, n = rand(g, T, H, BF16), torch.empty((T, H), dtype=BF16, device=DEV)
    r1, r2 = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    M.moe_block_norm(x, y, out, n, rstd_post=r1, rstd_pre=r2)
    want = ref.norm(x, y, None, None, None, 1.0, 1e-6, True, BF16, BF16)
    near(out, want["x_out"])
    near(n, want["n_out"])
    dn, dy, cols = rand(g, T, H, BF16), torch.empty((T, H), dtype=BF16, device=DEV), torch.empty(H, device=DEV)
    ws = torch.empty(M.moe_block_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    want = ref.norm_grad(x, dn, out, y, None, None, None, 1.0, r1, r2, True, BF16, BF16)
    dx = x  # in place
    M.moe_block_norm_backward(x, dn, out, y, dx, dy, ws, rstd_post=r1, rstd_pre=r2, dgamma_pre=cols)
    for name, got in (("dx", dx), ("dy", dy), ("dgamma_pre", cols)):
        near(got, want[name], name)
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, 1)[1].to(torch.int32).contiguous()
    offsets, perm = group(ids, E)
    w = dw = torch.rand((T, k), generator=g, device=DEV)
    wr = rand(g, E, H, BF16)
    dl, dwr, db = torch.empty((T, k), device=DEV), torch.empty((E, H), device=DEV), torch.empty(E, device=DEV)
    ws = torch.empty(M.moe_route_backward_workspace_size(T, k, E, H), dtype=torch.uint8, device=DEV)
    want = ref.route_grad(dw, w, ids, x, wr, None, BF16)
    M.moe_route_backward(dw, w, ids, x, wr, offsets, perm, dl, out, dwr, db, ws)
    for name, got in (("dlogits", dl), ("dx", out), ("dw_router", dwr), ("dbias", db)):
        near(got, want[name], name)
