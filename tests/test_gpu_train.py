"""The calls of a training step together: MoETrainLayer against the layer's definition in 64 bits, and its gradients
against differences."""
import pytest
import torch

import ffn_reference as ref
from sparse_moe_routed_gb300 import MoETrainLayer

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def layer(seed, T, H, E, k, I, keep, dw_type=F32, bias=True, T_max=None, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(shape, scale):
        return torch.randn(shape, generator=g, device=DEV) * scale

    wr = normal((E, H), 1 / H ** 0.5).to(BF16)
    b = normal((E,), 0.1) if bias else None
    wgu, wd = normal((E, 2 * I, H), std / H ** 0.5).to(BF16), normal((E, H, I), std / I ** 0.5).to(BF16)
    m = MoETrainLayer(wr, b, wgu, wd, k, T_max or T, keep=keep, dw_type=dw_type)
    return m, normal((T, H), 1.0).to(BF16), normal((T, H), 1.0).to(BF16)


def definition(m, x, ids):
    """The layer's output in 64 bits for the given routes, from float64 leaves."""
    leaves = [t.double().requires_grad_() for t in (x, m.w_router, m.w_gateup, m.w_down)]
    xx, wr, wgu, wd = leaves
    logits = xx @ wr.t()
    if m.bias is not None:
        leaves.append(m.bias.double().requires_grad_())
        logits = logits + leaves[-1]
    w = torch.softmax(logits.gather(1, ids), 1)
    out = torch.zeros_like(xx)
    for e in range(m.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        a = xx[t] @ wgu[e].t()
        g, u = a[:, :m.I], a[:, m.I:]
        y = (g * torch.sigmoid(g) * u) @ wd[e].t()
        out = out.index_add(0, t, w[t, j, None] * y)
    return out, leaves


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


# Each bf16 rounding moves a value by at most 2^-8 of it, at random by 2^-8 / sqrt(3) in the mean at most; a chain of n
# of them moves a sum of many such values by sqrt(n) times that.  An 8-bit value is off by half a step of at most
# amax / 63.5 (uniformly: that / sqrt(12)) where amax of 32 normal values is below 4 of their deviations: 4 / 63.5 /
# sqrt(12) = 0.018 of a value each, for g, u and x, and g's enters h' and the slope as well.
RND = 2.0 ** -8 / 3 ** 0.5
Q8 = 4 / 63.5 / 12 ** 0.5


@pytest.mark.parametrize("keep", ["q8", "bf16"])
@pytest.mark.parametrize("T,H,E,k,I", [(1, 128, 4, 2, 64), (16, 256, 64, 4, 64), (33, 256, 8, 3, 128),
                                       (300, 384, 16, 4, 192), (700, 256, 2, 1, 64)])
def test_step_against_the_definition(T, H, E, k, I, keep):
    m, x, dout = layer(T + H, T, H, E, k, I, keep, T_max=T + 5)
    out, dx = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    m.forward(x, out)
    want, leaves = definition(m, x, m.ids[:T].long())
    assert off(out, want) <= 4 * RND  # h, y, and their sum's terms
    want.backward(dout.double())
    add = torch.randn((T, H), device=DEV)
    m.backward(dout, dx, add=add)
    assert m.read_status() == 0
    tol = 6 * RND + (4 * Q8 if keep == "q8" else 2 * RND)
    assert off(dx - add, leaves[0].grad) <= tol
    for got, leaf in ((m.dw_gateup, leaves[2]), (m.dw_down, leaves[3])):
        assert off(got, leaf.grad) <= tol
    if k > 1:  # with one route the weight is 1 whatever the logits are
        assert off(m.dw_router, leaves[1].grad) <= tol and off(m.dbias, leaves[4].grad) <= tol


def test_gradients_against_differences():
    """The loss's change along a direction, of the layer as it runs (bf16 values kept).

    The direction is the gradient's, 1/100 of the weights' size: about 2.5 steps of bf16 (what it became is measured).
    Around 16 tokens an expert, and gradients of about 1, it moves a pre-activation by 0.01 / 16 * 256 * |dg|, under
    0.1, so that the third-order term of the difference is below 0.1^2 / 6 of it; the 16,384 outputs' roundings add
    about 0.5 to a change of some 100.
    """
    T, H, E, k, I = 64, 256, 8, 2, 64
    m, x, dout = layer(5, T, H, E, k, I, "bf16")
    out, dx = torch.empty((T, H), device=DEV), torch.empty((T, H), device=DEV)
    m.forward(x, out)
    ids = m.ids[:T].clone()
    m.backward(dout, dx)
    grads = {"w_gateup": m.dw_gateup.clone(), "w_down": m.dw_down.clone()}
    for name, grad in grads.items():
        w = getattr(m, name)
        old = w.clone()
        d = (grad * (0.01 * old.float().std() / grad.std())).to(BF16).float()
        loss = []
        for sign in (1, -1):
            w.copy_((old.float() + sign * d).to(BF16))
            m.forward(x, out)
            assert torch.equal(m.ids[:T], ids)
            loss.append((float((out.double() * dout.double()).sum()), w.float() - old.float()))
            w.copy_(old)
        (up, du), (down, dd) = loss
        want = float((grad.double() * (du - dd).double()).sum())
        assert abs((up - down) - want) <= 0.02 * abs(want)


def test_accumulated_micro_batches():
    T, H, E, k, I = 48, 256, 8, 2, 64
    m, x, dout = layer(9, T, H, E, k, I, "q8")
    out, dx = torch.empty((T, H), device=DEV, dtype=BF16), torch.empty((T, H), device=DEV, dtype=BF16)
    parts = []
    for s in (slice(0, 17), slice(17, 48)):
        m.forward(x[s], out[s])
        m.backward(dout[s], dx[s])
        parts.append((m.dw_gateup.clone(), m.dw_down.clone()))
    for i, s in enumerate((slice(0, 17), slice(17, 48))):
        m.forward(x[s], out[s])
        m.backward(dout[s], dx[s], accumulate=i > 0)
    assert torch.equal(m.dw_gateup, parts[0][0] + parts[1][0]) and torch.equal(m.dw_down, parts[0][1] + parts[1][1])


def test_step_in_a_graph():
    T, H, E, k, I = 40, 256, 16, 4, 64
    m, x, dout = layer(13, T, H, E, k, I, "q8", dw_type=BF16)
    out, dx = torch.empty((T, H), device=DEV, dtype=BF16), torch.empty((T, H), device=DEV, dtype=BF16)

    def step():
        m.forward(x, out)
        m.backward(dout, dx)

    step()
    got = lambda: [t.clone() for t in (out, dx, m.dw_router, m.dbias, m.dw_gateup, m.dw_down)]  # noqa: E731
    want = got()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (out, dx, m.dw_router, m.dbias, m.dw_gateup, m.dw_down):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got()))


def test_kept_bytes():
    """8 bits keep 33/64 of what bf16 does, of tokens and of gate and up values."""
    a, *_ = layer(1, 16, 256, 8, 2, 64, "q8")
    b, *_ = layer(1, 16, 256, 8, 2, 64, "bf16")
    small = sum(t.nbytes for t in (a.x, a.x_exp, a.act, a.act_exp))
    assert 64 * small == 33 * sum(t.nbytes for t in (b.x, b.act))
