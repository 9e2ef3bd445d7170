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
