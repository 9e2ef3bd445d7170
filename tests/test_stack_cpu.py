"""MoEStack's host side without a GPU: which calls it binds, and what it refuses.

The calls are built and looked at, never issued: a layer is a stand-in that
holds an output buffer, and the stream is a number.
"""
from types import SimpleNamespace

import pytest
import torch

from sparse_moe_routed_gb300 import MoEStack

H = 128
STREAM = SimpleNamespace(cuda_stream=0)


class Layer:
    def __init__(self, T_max, H=H):
        self.H, self.T_max = H, T_max
        self.w_router = torch.empty((4, H), dtype=torch.bfloat16)
        self.out = torch.empty((T_max, H), dtype=torch.bfloat16)

    def bound_calls(self, x, T=None, out=None, stream=None, residual=None, out_f32=None, route=True):
        return [("layer", None, (T,))]


def stack(T_max=8, layers=2, **kw):
    return MoEStack([Layer(T_max) for _ in range(layers)], T_max, **kw)


@pytest.mark.parametrize("kw", [{}, {"scale": 0.5}], ids=["plain", "norms after the layers"])
def test_streams_that_the_buffers_do_not_hold_are_refused(kw):
    s = stack(**kw)
    for T in (1, 7, 8):
        assert len(s.layer_calls(torch.zeros((T, H)), 0, STREAM)) >= 2
    for x in (torch.zeros((9, H)), torch.zeros((8, H + 1)), torch.zeros((8, 2 * H)), torch.zeros((8, H // 2)),
              torch.zeros((8, H), dtype=torch.bfloat16), torch.zeros((8, H), dtype=torch.float64),
              torch.zeros((H, 8)).t(), torch.zeros((8, 2 * H))[:, :H], torch.zeros(H)):
        with pytest.raises(AssertionError):
            s.layer_calls(x, 0, STREAM)


@pytest.mark.parametrize("kw", [{}, {"scale": 0.5}], ids=["plain", "norms after the layers"])
def test_a_layer_smaller_than_the_stack_is_refused_before_the_first_call(kw):
    s = MoEStack([Layer(8), Layer(4)], 8, **kw)
    assert s.layer_calls(torch.zeros((4, H)), 1, STREAM)
    with pytest.raises(AssertionError):
        s.layer_calls(torch.zeros((5, H)), 1, STREAM)
    with pytest.raises(AssertionError):  # before anything of layer 0 is issued
        s.forward(torch.zeros((5, H)), STREAM)


def test_layers_of_different_widths_are_refused():
    with pytest.raises(AssertionError):
        MoEStack([Layer(8), Layer(8, 2 * H)], 8)


@pytest.mark.parametrize("name", ["post_gammas", "gates"])
def test_one_vector_per_layer(name):
    stack(**{name: [None, None]})
    stack(**{name: [torch.zeros(H), None]})
    for n in (0, 1, 3):
        with pytest.raises(AssertionError):
            stack(**{name: [None] * n})


def test_vectors_of_another_shape_type_or_device_are_refused():
    stack(gates=[None, torch.zeros((8, 1))])
    bad = [torch.zeros(H - 1), torch.zeros(H, dtype=torch.bfloat16), torch.zeros(2 * H)[::2],
           torch.zeros(H, device="meta")]
    for name, more in (("post_gammas", [torch.zeros((8, 1))]), ("gates", [torch.zeros((7, 1)), torch.zeros((8, 2))])):
        for v in bad + more:
            with pytest.raises(AssertionError):
                stack(**{name: [None, v]})
    # one list for both: a gate per token is no gain
    both = [torch.zeros((8, 1))] * 2
    with pytest.raises(AssertionError):
        stack(post_gammas=both, gates=both)


def bound(s, x, l=0, nxt=1):
    """The arguments of the norm before layer l and of the norms after it."""
    calls = {c[0]: c[2] for c in s.layer_calls(x, l, STREAM, nxt=nxt)}
    plain = [v.value if hasattr(v, "value") else v for v in calls["moe_rmsnorm"]]
    return plain, [v.value if hasattr(v, "value") else v for v in calls["moe_block_norm"]]


def test_replaced_vectors_scale_and_eps_reach_the_next_call():
    """A per-token gate is new with every batch: the calls of one stream buffer follow the stack's attributes."""
    vec = lambda: [torch.zeros(H) for _ in range(2)]
    s, x = stack(gammas=vec(), post_gammas=vec(), gates=vec()), torch.zeros((8, H))
    bound(s, x)
    s.gates[0] = torch.zeros((8, 1))
    s.post_gammas[0], s.gammas[0], s.gammas[1] = torch.zeros(H), torch.zeros(H), torch.zeros(H)
    s.scale, s.eps = 0.5, 1e-3
    s.layers[0].out = torch.empty((8, H), dtype=torch.bfloat16)
    before, after = bound(s, x)
    assert before[1] == s.gammas[0].data_ptr() and abs(before[2] - 1e-3) < 1e-9
    assert after[3] == s.layers[0].out.data_ptr()
    assert (after[6], after[7]) == (s.gates[0].data_ptr(), 2)  # per token
    assert (after[9], after[10]) == (s.post_gammas[0].data_ptr(), s.gammas[1].data_ptr())
    assert after[12] == 0.5 and abs(after[13] - 1e-3) < 1e-9
    s.gates[0] = None
    assert bound(s, x)[1][6:8] == [None, 0]
    s.gates = None
    assert bound(s, x)[1][6:8] == [None, 0]


def test_norms_after_the_layers_may_be_asked_for_later():
    s, x = stack(), torch.zeros((8, H))
    assert [c[0] for c in s.layer_calls(x, 0, STREAM)] == ["moe_rmsnorm", "layer"]
    s.scale = 0.5
    assert bound(s, x)[1][12] == 0.5


def test_a_replaced_vector_is_checked():
    s, x = stack(gammas=[None, None], gates=[None, None], post_gammas=[None, None]), torch.zeros((8, H))
    bound(s, x)
    for name in ("gammas", "gates", "post_gammas"):
        for v in (torch.zeros(H - 1), torch.zeros(H, dtype=torch.bfloat16), torch.zeros(2 * H)[::2]):
            getattr(s, name)[0] = v
            with pytest.raises(AssertionError):
                s.layer_calls(x, 0, STREAM)
        getattr(s, name)[0] = None
    assert bound(s, x)


def test_raw_without_the_norm_that_writes_it_is_refused():
    s, x, raw = stack(scale=0.5), torch.zeros((8, H)), torch.zeros((8, H), dtype=torch.bfloat16)
    assert s.layer_calls(x, 0, STREAM, raw=raw)[0][2][6].value == raw.data_ptr()
    with pytest.raises(AssertionError):
        s.layer_calls(x, 1, STREAM, raw=raw, first=False)
    # without norms after the layers every layer has its own norm before it
    assert stack().layer_calls(x, 1, STREAM, raw=raw, first=False)[0][2][6].value == raw.data_ptr()
