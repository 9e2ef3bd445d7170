"""MoEStack's norms after the layers and the launch forms of libmoe_block that
only larger calls reach, against the definitions in 64 bits."""
import pytest
import torch

import sparse_moe_routed_gb300 as M
import workloads as wl

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
