"""Host side of the experts' training operators without a GPU: refusals, and the tests' reference gradients against
differences of the definition."""
import ctypes as C

import pytest
import torch

import ffn_reference as ref
from sparse_moe_routed_gb300 import MoEError, _block, _lib
import sparse_moe_routed_gb300 as M

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: CPU-only host checks")

A = [C.c_void_p((1 << 20) + (i << 16)) for i in range(24)]
ODD, EIGHT = C.c_void_p((1 << 20) + 1), C.c_void_p((1 << 20) + 8)
F32, BF16 = _block.MOE_ROW_F32, _block.MOE_ROW_BF16
EINVAL, ESHAPE, ENOTSUP, EWS = _lib.MOE_EINVAL, _lib.MOE_ESHAPE, _lib.MOE_ENOTSUP, _lib.MOE_EWORKSPACE

SAVE = [("x", A[0]), ("ldx", 64), ("type", BF16), ("T", 16), ("H", 64), ("q", A[1]), ("ldq", 64), ("e", A[2]),
        ("lde", 2), ("stream", None)]
LOAD = [("q", A[0]), ("ldq", 64), ("e", A[1]), ("lde", 2), ("T", 16), ("H", 64), ("inv", A[2]), ("w", A[3]), ("k", 4),
        ("R", 64), ("out", A[4]), ("ldo", 64), ("type", BF16), ("status", None), ("stream", None)]
FFN = [("x", A[0]), ("ldx", 64), ("wgu", A[1]), ("wd", A[2]), ("off", A[3]), ("R", 16), ("E", 4), ("H", 64), ("I", 32),
       ("h", A[4]), ("act", A[5]), ("kind", _block.MOE_ACT_Q8), ("lda", 64), ("e", A[6]), ("lde", 2), ("y", A[7]),
       ("ldy", 64), ("ytype", F32), ("status", None), ("stream", None)]
FFN_B = [("dy", A[0]), ("lddy", 64), ("x", A[1]), ("ldx", 64), ("act", A[2]), ("kind", _block.MOE_ACT_Q8), ("lda", 64),
         ("e", A[3]), ("lde", 2), ("wgu", A[4]), ("wd", A[5]), ("off", A[6]), ("R", 16), ("E", 4), ("H", 64), ("I", 32),
         ("dx", A[7]), ("lddx", 64), ("dxtype", F32), ("dwgu", A[8]), ("dwd", A[9]), ("dwtype", F32), ("acc", 0),
         ("ws", A[10]), ("wsb", 1 << 20), ("status", None), ("stream", None)]
CALLS = {"moe_checkpoint_save": SAVE, "moe_checkpoint_load": LOAD, "moe_ffn": FFN, "moe_ffn_backward": FFN_B}

save, load, ffn, ffn_b = CALLS
REFUSALS = [
    (save, dict(x=None), EINVAL), (save, dict(q=None), EINVAL), (save, dict(e=None), EINVAL), (save, dict(x=ODD), EINVAL),
    (save, dict(type=2), EINVAL), (save, dict(q=A[0]), EINVAL), (save, dict(e=A[1]), EINVAL), (save, dict(T=-1), ESHAPE),
    (save, dict(H=0), ESHAPE), (save, dict(ldx=63), ESHAPE), (save, dict(ldq=63), ESHAPE), (save, dict(lde=1), ESHAPE),
    (save, dict(H=65537, ldx=1 << 17, ldq=1 << 17, lde=1 << 17), ENOTSUP), (save, dict(T=(1 << 30) + 1), ENOTSUP),
    (save, dict(ldq=1 << 60), ENOTSUP), (save, dict(ldx=1 << 60), ENOTSUP), (save, dict(lde=1 << 60), ENOTSUP),
    (load, dict(q=None), EINVAL), (load, dict(e=None), EINVAL), (load, dict(out=None), EINVAL),
    (load, dict(inv=None), EINVAL), (load, dict(inv=ODD), EINVAL), (load, dict(w=ODD), EINVAL),
    (load, dict(out=ODD), EINVAL), (load, dict(out=A[0]), EINVAL), (load, dict(type=-1), EINVAL),
    (load, dict(status=ODD), EINVAL), (load, dict(k=0), ESHAPE), (load, dict(R=-1), ESHAPE), (load, dict(ldo=63), ESHAPE),
    (load, dict(k=33), ENOTSUP), (load, dict(T=1 << 29), ENOTSUP),
    (ffn, dict(x=None), EINVAL), (ffn, dict(wgu=None), EINVAL), (ffn, dict(wd=None), EINVAL), (ffn, dict(off=None), EINVAL),
    (ffn, dict(h=None), EINVAL), (ffn, dict(act=None), EINVAL), (ffn, dict(e=None), EINVAL), (ffn, dict(kind=3), EINVAL),
    (ffn, dict(kind=0), EINVAL), (ffn, dict(x=EIGHT), EINVAL), (ffn, dict(wgu=EIGHT), EINVAL), (ffn, dict(wd=EIGHT), EINVAL),
    (ffn, dict(h=EIGHT), EINVAL), (ffn, dict(y=EIGHT), EINVAL), (ffn, dict(off=ODD), EINVAL), (ffn, dict(y=A[0]), EINVAL),
    (ffn, dict(h=A[7]), EINVAL), (ffn, dict(act=A[4]), EINVAL), (ffn, dict(ytype=2), EINVAL), (ffn, dict(ldx=68), EINVAL),
    (ffn, dict(kind=1, lda=68), EINVAL), (ffn, dict(R=-1), ESHAPE), (ffn, dict(E=0), ESHAPE), (ffn, dict(H=0), ESHAPE),
    (ffn, dict(I=-8), ESHAPE), (ffn, dict(ldx=56), ESHAPE), (ffn, dict(lda=63), ESHAPE), (ffn, dict(lde=1), ESHAPE),
    (ffn, dict(ldy=8), ESHAPE), (ffn, dict(H=60), ENOTSUP), (ffn, dict(I=36), ENOTSUP), (ffn, dict(E=1025), ENOTSUP),
    (ffn, dict(H=65544, ldx=1 << 17, ldy=1 << 17), ENOTSUP), (ffn, dict(R=(1 << 30) + 1), ENOTSUP),
    (ffn_b, dict(dy=None), EINVAL), (ffn_b, dict(x=None), EINVAL), (ffn_b, dict(act=None), EINVAL),
    (ffn_b, dict(e=None), EINVAL), (ffn_b, dict(kind=0), EINVAL), (ffn_b, dict(wgu=None), EINVAL),
    (ffn_b, dict(wd=None), EINVAL), (ffn_b, dict(off=None), EINVAL), (ffn_b, dict(dx=A[0]), EINVAL),
    (ffn_b, dict(dwd=A[8]), EINVAL), (ffn_b, dict(dx=None, dwgu=None, dwd=None), EINVAL), (ffn_b, dict(ws=None), EWS),
    (ffn_b, dict(wsb=16 * 3 * 32 * 2 + 15), EWS), (ffn_b, dict(ws=EIGHT), EINVAL), (ffn_b, dict(ws=A[7]), EINVAL),
    (ffn_b, dict(dwgu=C.c_void_p((1 << 20) + 16)), EINVAL), (ffn_b, dict(dxtype=5), EINVAL), (ffn_b, dict(dwtype=2), EINVAL),
    (ffn_b, dict(lddy=8), ESHAPE), (ffn_b, dict(I=12), ENOTSUP), (ffn_b, dict(R=-1), ESHAPE),
    (ffn, dict(ldx=1 << 38), ENOTSUP), (ffn_b, dict(lddy=1 << 38), ENOTSUP), (ffn_b, dict(ldx=1 << 38), ENOTSUP),
]


@no_gpu
@pytest.mark.parametrize("name,change,want", REFUSALS, ids=[f"{n}-{list(c.items())[0]}-{i}" for i, (n, c, _) in enumerate(REFUSALS)])
def test_refused_on_the_host(name, change, want):
    spec = CALLS[name]
    assert set(change) <= {k for k, _ in spec}
    assert getattr(_block.load(), name)(*[change.get(k, v) for k, v in spec]) == want


def test_workspace_size():
    """dg and du, h, and a word for the queue of tiles, in whole 16 bytes."""
    assert M.moe_ffn_backward_workspace_size(5, 8) == 240 + 16
    assert M.moe_ffn_backward_workspace_size(1, 8) == 48 + 16
    assert M.moe_ffn_backward_workspace_size(40960, 640) == 40960 * 640 * 6 + 16
    assert M.moe_ffn_backward_workspace_size(1 << 20, 65536) == (1 << 36) * 6 + 16
    assert M.moe_ffn_backward_workspace_size(-1, 8) == 0 == M.moe_ffn_backward_workspace_size(1, 0)


def test_tensors_on_the_cpu_are_refused():
    x = torch.zeros((2, 8), dtype=torch.bfloat16)
    with pytest.raises(MoEError):
        M.moe_checkpoint_save(x, x.to(torch.int8), torch.zeros((2, 1), dtype=torch.uint8))
    with pytest.raises(MoEError):
        M.moe_ffn(x, torch.zeros((1, 16, 8), dtype=torch.bfloat16), torch.zeros((1, 8, 8), dtype=torch.bfloat16),
                  torch.zeros(2, dtype=torch.int32), x, x.clone())


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    n, H, I = 5, 7, 6
    x, wgu, wd, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((n, H), (2 * I, H), (H, I), (n, H)))

    def loss(x, wgu, wd):
        a = x @ wgu.t()
        z = a[:, :I]
        return ((z / (1 + torch.exp(-z)) * a[:, I:]) @ wd.t() * dy).sum()

    a = x @ wgu.t()
    got = ref.backward(dy, x, a[:, :I], a[:, I:], wgu, wd, torch.float64, torch.float64)
    for i, name in enumerate(("dx", "dwgu", "dwd")):
        args = [x, wgu, wd]
        want = torch.zeros_like(args[i])
        for j in range(args[i].numel()):
            step = torch.zeros_like(args[i])
            step.view(-1)[j] = 1e-6
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + step, args[i] - step
            want.view(-1)[j] = (loss(*up) - loss(*down)) / 2e-6
        assert torch.allclose(got[name][0], want, rtol=1e-6, atol=1e-7), name


def test_reference_of_8_bits():
    """The smallest power of two that fits, by trying them all."""
    g = torch.Generator().manual_seed(4)
    x = (torch.randn((200, 40), generator=g) * torch.exp(3 * torch.randn((200, 1), generator=g))).double()
    x[0, :32], x[1, :32], x[2, :32] = 127.0, 127.5, 0.0
    q, e = ref.quantise(x)
    for r in range(200):
        for c in (0, 32):
            v = x[r, c:c + 32]
            k = -126
            while float(v.abs().max()) > 127 * 2.0 ** k:
                k += 1
            assert int(e[r, c // 32]) == k + 127
            assert torch.equal(q[r, c:c + 32].double(), torch.round(v / 2.0 ** k))
    assert torch.equal(ref.values(q, e).to(torch.bfloat16).double(), ref.values(q, e))  # bf16 numbers
