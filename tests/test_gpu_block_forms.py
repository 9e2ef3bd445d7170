"""MoEStack's norms after the layers and the launch forms of libmoe_block that
only larger calls reach, against the definitions in 64 bits."""
import pytest
import torch

import block_reference as ref
import sparse_moe_routed_gb300 as M
import workloads as wl
from sparse_moe_routed_gb300 import _lib, pack_layer_experts
from test_gpu_block import group, near, rand

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
