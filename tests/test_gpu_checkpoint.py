"""Activations in 8 bits on the GPU: the same bits as the definition in 64 bits."""
import pytest
import torch

import ffn_reference as ref
import sparse_moe_routed_gb300 as M
from sparse_moe_routed_gb300 import MoEError

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def view(n, H, dtype, pad=0, shift=0, fill=7):
    buf = torch.full((n * (H + pad) + shift + 8,), fill, dtype=dtype, device=DEV)
    return torch.as_strided(buf, (n, H), (H + pad, 1), shift), buf


def rest_is(buf, v, fill=7):
    mask = torch.ones(buf.shape, dtype=torch.bool, device=DEV)
    torch.as_strided(mask, v.shape, v.stride(), v.storage_offset()).fill_(False)
    return bool((buf[mask] == fill).all())


def sample(g, T, H, dtype):
    """Values of all sizes, exact ties, groups of zeros and of the smallest numbers."""
    x = torch.randn((T, H), generator=g, device=DEV) * torch.exp(2 * torch.randn((T, H), generator=g, device=DEV))
    x = x * 2.0 ** torch.randint(-140, 120, (T, 1), generator=g, device=DEV).double()
    x = x.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)
    x[::5] = (torch.randint(-254, 255, (len(x[::5]), H), generator=g, device=DEV) / 2).to(dtype)
    x[::7] = 0
    return x


SIZES = [(1, 1), (1, 31), (2, 32), (3, 33), (5, 64), (16, 2560), (7, 1001), (509, 1001), (33, 1026), (4, 8200), (2, 65536),
         (1000, 8), (129, 264)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1), (2, 2)])
def test_there_and_back(T, H, pad, shift, dtype):
    g = gen(T * 31 + H + pad)
    x, _ = view(T, H, dtype, pad, shift)
    x.copy_(sample(g, T, H, dtype))
    G = -(-H // 32)
    q, qb = view(T, H, torch.int8, pad, shift)
    e, eb = view(T, G, torch.uint8, pad, shift)
    M.moe_checkpoint_save(x, q, e)
    wq, we = ref.quantise(x)
    assert torch.equal(q, wq) and torch.equal(e, we)
    assert rest_is(qb, q) and rest_is(eb, e)
    for t in (F32, BF16):
        y, yb = view(T, H, t, pad, shift)
        M.moe_checkpoint_load(q, e, y)
        assert torch.equal(y.double(), ref.values(q, e))  # nothing is rounded
        assert rest_is(yb, y)
    # half a step, less than amax / 127; at the top of the range a step
    amax = torch.nn.functional.pad(x.double().abs(), (0, G * 32 - H)).view(T, G, 32).amax(2).repeat_interleave(32, 1)[:, :H]
    off = (ref.values(q, e) - x.double()).abs()
    assert bool((off <= torch.where(amax <= 127 * 2.0 ** 121, amax / 127, amax / 126).clamp_min(2.0 ** -127)).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("T,H,k", [(1, 1, 1), (3, 33, 4), (16, 2560, 10), (700, 264, 32), (5, 1001, 6), (1200, 136, 3)])
@pytest.mark.parametrize("pad,shift,weighted", [(0, 0, False), (8, 0, True), (3, 1, False), (2, 2, True)])
def test_into_expert_order(T, H, k, pad, shift, weighted, dtype):
    g = gen(T + H + k)
    R = T * k + 5
    inv = torch.randperm(R, generator=g, device=DEV)[:T * k].to(torch.int32).view(T, k)
    inv = torch.where(torch.rand((T, k), generator=g, device=DEV) < 0.2, torch.full_like(inv, -1), inv).contiguous()
    w = torch.randn((T, k), generator=g, device=DEV) if weighted else None
    q, e = ref.quantise(torch.randn((T, H), generator=g, device=DEV))
    out, buf = view(R, H, dtype, pad, shift)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_checkpoint_load(q, e, out, inv_perm=inv, w=w, dev_status=st)
    # the same bits as reading back in token order and dispatching
    rows, want = torch.empty((T, H), dtype=dtype, device=DEV), torch.full((R, H), 7, dtype=dtype, device=DEV)
    M.moe_checkpoint_load(q, e, rows)
    M.moe_dispatch(rows, inv, want, w=w)
    assert torch.equal(out, want) and rest_is(buf, out) and int(st) == 0


def test_groups_with_nan_and_infinities():
    x = torch.ones((3, 100), device=DEV)
    x[0, 40], x[1, 70], x[2, 99] = float("nan"), float("inf"), -float("inf")
    q, e = torch.empty((3, 100), dtype=torch.int8, device=DEV), torch.empty((3, 4), dtype=torch.uint8, device=DEV)
    M.moe_checkpoint_save(x, q, e)
    want = torch.zeros((3, 100), dtype=torch.bool, device=DEV)
    want[0, 32:64], want[1, 64:96], want[2, 96:] = True, True, True
    for t in (F32, BF16):
        y = torch.empty((3, 100), dtype=t, device=DEV)
        M.moe_checkpoint_load(q, e, y)
        assert torch.equal(y.isnan(), want) and bool((y[~want] == 1).all())


def test_every_exponent_byte():
    e = torch.arange(256, dtype=torch.int32, device=DEV).to(torch.uint8).view(256, 1)
    q = torch.arange(256, device=DEV)[:, None].expand(256, 32).to(torch.int8).contiguous()
    q = (q + torch.arange(32, device=DEV, dtype=torch.int8)).contiguous()
    y = torch.empty((256, 32), device=DEV)
    M.moe_checkpoint_load(q, e, y)
    want = ref.values(q, e).float()
    assert torch.equal(y.nan_to_num(posinf=3e38, neginf=-3e38), want.nan_to_num(posinf=3e38, neginf=-3e38))
    assert bool(y[255].isnan().all())


def test_bad_slots_set_the_status():
    q, e = ref.quantise(torch.ones((2, 64), device=DEV))
    out = torch.zeros((4, 64), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    inv = torch.tensor([[0, 4], [-2, 3]], dtype=torch.int32, device=DEV)
    M.moe_checkpoint_load(q, e, out, inv_perm=inv, dev_status=st)
    assert int(st) == 1 and out[:, 0].tolist() == [1, 0, 0, 1]


def test_rows_past_32_bit_offsets():
    """The last rows of a matrix of more than 2^32 bytes."""
    T, H = 66000, 65536
    q = torch.zeros((T, H), dtype=torch.int8, device=DEV)
    e = torch.full((T, H // 32), 127, dtype=torch.uint8, device=DEV)
    x = torch.zeros((T, H), dtype=BF16, device=DEV)
    x[-2:] = 3
    M.moe_checkpoint_save(x, q, e)
    assert bool((e[-2:] == 127 - 5).all()) and bool((q[-2:] == 96).all()) and bool((q[-3] == 0).all())
    x.zero_()
    M.moe_checkpoint_load(q, e, x)
    assert bool((x[-2:] == 3).all()) and bool((x[-3] == 0).all())


def test_refusals_of_the_binding():
    x = torch.ones((4, 64), device=DEV)
    q, e = torch.empty((4, 64), dtype=torch.int8, device=DEV), torch.empty((4, 2), dtype=torch.uint8, device=DEV)
    inv = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    bad = [lambda: M.moe_checkpoint_save(x.double(), q, e), lambda: M.moe_checkpoint_save(x, q.float(), e),
           lambda: M.moe_checkpoint_save(x, q, e[:, :1]), lambda: M.moe_checkpoint_save(x, q[:3], e),
           lambda: M.moe_checkpoint_save(x.cpu(), q, e), lambda: M.moe_checkpoint_save(x.t(), q, e),
           lambda: M.moe_checkpoint_load(q, e, x[:3]), lambda: M.moe_checkpoint_load(q, e, x.double()),
           lambda: M.moe_checkpoint_load(q, e, x, w=torch.ones((4, 2), device=DEV)),
           lambda: M.moe_checkpoint_load(q, e, x, inv_perm=inv.long()),
           lambda: M.moe_checkpoint_load(q, e, x, inv_perm=inv[:3]),
           lambda: M.moe_checkpoint_load(q, e, x, inv_perm=inv, w=torch.ones((4, 3), device=DEV))]
    for i, call in enumerate(bad):
        with pytest.raises(MoEError):
            call()
            pytest.fail(f"call {i} was accepted")
