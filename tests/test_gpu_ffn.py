"""The experts' feed-forward block and its gradient on the GPU.

Twice: on whole numbers chosen so that every product, sum and rounding is exact
(the outputs have to be equal), and on random values against the definitions in
64 bits, inside the bounds of ffn_reference.py.
"""
import pytest
import torch

import ffn_reference as ref
import sparse_moe_routed_gb300 as M
from sparse_moe_routed_gb300 import MoEError

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
NAN = float("nan")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def matrix(n, w, dtype, pad=0, fill=NAN):
    return torch.full((n, w + pad), fill, dtype=dtype, device=DEV)[:, :w]


def offsets(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device=DEV), o


def groups(I):
    return -(-I // 32)


def near(got, want, name):
    value, bound = want
    off = (got.to(F64) - value).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst {float((off - bound).max()):.3e}"


def keep(kind, R, I, pad=0):
    """Buffers for gate and up values."""
    if kind == "none":
        return None, None
    if kind == "bf16":
        return matrix(R, 2 * I, BF16, 8 * pad), None
    q = torch.full((R, 2 * I + pad), 77, dtype=torch.int8, device=DEV)[:, :2 * I]
    return q, torch.full((R, 2 * groups(I) + pad), 1, dtype=torch.uint8, device=DEV)[:, :2 * groups(I)]


class Block:
    """Weights and rows of a block; rows outside the experts' hold NaN."""

    def __init__(self, counts, H, I, seed, whole, behind=3, first=0, pad=0):
        g = gen(seed)
        self.counts, self.H, self.I, self.E = counts, H, I, len(counts)
        self.off, self.o = offsets(counts, first)
        self.R = R = self.o[-1] + behind
        self.x, self.dy = matrix(R, H, BF16, pad), matrix(R, H, BF16, pad)
        rows = slice(first, self.o[-1])
        n = self.o[-1] - first

        def ints(shape, share, lo=-1, hi=1):
            v = torch.randint(lo, hi + 1, shape, generator=g, device=DEV).float()
            return torch.where(torch.rand(shape, generator=g, device=DEV) < share, v, torch.zeros_like(v))

        E = self.E
        if whole:
            # few nonzero inputs, so that sums stay whole numbers of at most 8 bits where bf16 has to hold them
            few = min(1.0, 12 / H)
            self.wgu = torch.cat([128 * ints((E, I, H), 0.8), ints((E, I, H), 0.8)], 1).to(BF16)
            self.wd = ints((E, H, I), 0.8).to(BF16)
            self.x[rows] = ints((n, H), few).to(BF16)
            self.dy[rows] = ints((n, H), few).to(BF16)
        else:
            self.wgu = (torch.randn((E, 2 * I, H), generator=g, device=DEV) / H ** 0.5).to(BF16)
            self.wd = (torch.randn((E, H, I), generator=g, device=DEV) / I ** 0.5).to(BF16)
            self.x[rows] = torch.randn((n, H), generator=g, device=DEV).to(BF16)
            self.dy[rows] = torch.randn((n, H), generator=g, device=DEV).to(BF16)
        self.g = g

    def experts(self):
        return [(e, slice(self.o[e], self.o[e + 1])) for e in range(self.E) if self.counts[e]]

    def outside(self):
        m = torch.ones(self.R, dtype=torch.bool, device=DEV)
        m[self.o[0]:self.o[-1]] = False
        return m

    def kept(self, kind, whole):
        """Gate and up values as a forward pass could have kept them."""
        R, I, g = self.R, self.I, self.g
        if whole:  # 64: its sigmoid is 1 in fp32; 0: one half, and no up gradient; u small
            gate = 64.0 * torch.randint(0, 2, (R, I), generator=g, device=DEV)
            up = torch.randint(-1, 2, (R, I), generator=g, device=DEV).float() * 2
        else:
            gate, up = (2 * torch.randn((R, I), generator=g, device=DEV) for _ in range(2))
        a, e = keep(kind, R, I, 1)
        out = self.outside()
        if kind == "bf16":
            a[:, :I], a[:, I:] = gate.to(BF16), up.to(BF16)
            a[out] = NAN
        else:
            for k, v in enumerate((gate, up)):
                q, x = ref.quantise(v)
                a[:, k * I:(k + 1) * I], e[:, k * groups(I):(k + 1) * groups(I)] = q, x
            e[out] = 255
        return a, e


SHAPES = [  # rows of each expert, H, I
    ([1], 8, 8), ([3], 16, 8), ([1, 0, 2], 64, 32), ([16, 17, 15], 72, 40), ([0, 0, 5], 128, 64), ([0], 64, 64),
    ([31, 32, 33, 0, 64], 136, 24), ([65, 1, 127], 256, 64), ([128, 129], 264, 136), ([255, 256, 257], 320, 200),
    ([513, 2], 512, 264), ([7, 300, 80, 0, 1], 1000, 200), ([96, 20], 2560, 640), ([1, 2, 1, 4], 2560, 640),
    ([600], 520, 1032), ([2, 700, 1, 0, 33, 64, 48, 16], 192, 320),
]
ids = [f"{'+'.join(map(str, c))}-{H}x{I}" for c, H, I in SHAPES]


@pytest.mark.parametrize("kind", ["none", "bf16", "q8"])
@pytest.mark.parametrize("counts,H,I", SHAPES, ids=ids)
def test_forward_on_whole_numbers(counts, H, I, kind):
    b = Block(counts, H, I, H + I, True, first=2, pad=8)
    h, y = matrix(b.R, I, BF16), matrix(b.R, H, F32, 8)
    a, e = keep(kind, b.R, I, 3)
    before = a.clone() if a is not None else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=a, act_exp=e, dev_status=st)
    assert int(st) == 0
    for k, s in b.experts():
        x, wgu, wd = b.x[s].double(), b.wgu[k].double(), b.wd[k].double()
        g, u = x @ wgu[:I].t(), x @ wgu[I:].t()
        assert float((g / 128).abs().max()) <= 127 and float(u.abs().max()) <= 127
        if kind != "none":
            gg, uu = ref.act_values(a[s], e[s] if e is not None else None)
            assert torch.equal(gg, g) and torch.equal(uu, u)
        hh = g.clamp_min(0) * u  # silu of 128 n: itself or nothing
        assert torch.equal(h[s].double(), hh.to(BF16).double())
        want = hh.to(BF16).double() @ wd.t()
        assert float(want.abs().max()) < 2 ** 24
        assert torch.equal(y[s].double(), want)
    out = b.outside()
    assert bool(h[out].isnan().all()) and bool(y[out].isnan().all())
    if kind == "bf16":
        assert bool(a[out].isnan().all())
    elif kind == "q8":
        assert torch.equal(a[out], before[out]) and bool((e[out] == 1).all())


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("counts,H,I", SHAPES, ids=ids)
def test_backward_on_whole_numbers(counts, H, I, kind):
    b = Block(counts, H, I, 3 * H + I, True, first=1, pad=8)
    a, e = b.kept(kind, True)
    dx = matrix(b.R, H, F32, 8)
    dwgu, dwd = (torch.full(w.shape, NAN, device=DEV) for w in (b.wgu, b.wd))
    ws = torch.full((M.moe_ffn_backward_workspace_size(b.R, I),), 255, dtype=torch.uint8, device=DEV)  # NaN
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx, dwgu, dwd, ws, act_exp=e, dev_status=st)
    assert int(st) == 0
    want_gu, want_d = torch.zeros_like(dwgu, dtype=F64), torch.zeros_like(dwd, dtype=F64)
    for k, s in b.experts():
        g, u = ref.act_values(a[s], e[s] if e is not None else None)
        dy, x = b.dy[s].double(), b.x[s].double()
        dh = dy @ b.wd[k].double()
        assert float(dh.abs().max()) <= 127
        r = torch.where(g > 0, 1.0, 0.5)
        da = torch.cat([dh * u * r, dh * g * r], 1)
        want = da @ b.wgu[k].double()
        assert torch.equal(dx[s].double(), want) and float(want.abs().max()) < 2 ** 24
        want_gu[k] = da.t() @ x
        want_d[k] = dy.t() @ (g * r * u)
    assert torch.equal(dwgu.double(), want_gu)
    assert torch.equal(dwd.double(), want_d)
    assert bool(dx[b.outside()].isnan().all())
    # added to what is there, and in bf16
    M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, None, dwgu, None, ws, act_exp=e, accumulate=True)
    M.moe_ffn_backward(b.dy, None, a, None, b.wd, b.off, None, None, dwd, ws, act_exp=e, accumulate=True)
    assert torch.equal(dwgu.double(), 2 * want_gu) and torch.equal(dwd.double(), 2 * want_d)
    dx16, dwgu16, dwd16 = matrix(b.R, H, BF16, 16), torch.full_like(b.wgu, 1.0), torch.full_like(b.wd, NAN)
    M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx16, dwgu16, None, ws, act_exp=e, accumulate=True)
    M.moe_ffn_backward(b.dy, None, a, None, b.wd, b.off, None, None, dwd16, ws, act_exp=e)
    for k, s in b.experts():
        assert torch.equal(dx16[s], dx[s].to(BF16))
    assert torch.equal(dwgu16, (1 + want_gu.float()).to(BF16)) and torch.equal(dwd16, want_d.float().to(BF16))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("counts,H,I", SHAPES, ids=ids)
def test_forward_on_random_values(counts, H, I, dtype):
    b = Block(counts, H, I, 5 * H + I, False)
    h, y = matrix(b.R, I, BF16), matrix(b.R, H, dtype)
    a, _ = keep("bf16", b.R, I)
    M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=a)
    q, qe = keep("q8", b.R, I)
    h2, y2 = matrix(b.R, I, BF16), matrix(b.R, H, dtype)
    M.moe_ffn(b.x, b.wgu, b.wd, b.off, h2, y2, act=q, act_exp=qe)
    for k, s in b.experts():
        want = ref.forward(b.x[s], b.wgu[k], b.wd[k], dtype)
        for j, n in enumerate("gu"):
            v, vb = want[n]
            near(a[s, j * I:(j + 1) * I], ref.out(v, vb, BF16), n)
            # in 8 bits: half a step of the group's scale, which is at most amax / 63.5
            G = groups(I)
            got = ref.values(q[s, j * I:(j + 1) * I], qe[s, j * G:(j + 1) * G])
            pad = torch.nn.functional.pad(v.abs() + vb, (0, G * 32 - I)).view(len(v), G, 32).amax(2)
            step = (pad / 63.5).repeat_interleave(32, 1)[:, :I]
            near(got, (v, 1.1 * vb + step / 2), n + " in 8 bits")
        near(h[s], want["h"], "h")
        near(y[s], want["y"], "y")
        assert torch.equal(h[s], h2[s]) and torch.equal(y[s], y2[s])


@pytest.mark.parametrize("kind,dx_type,dw_type", [("bf16", BF16, F32), ("q8", F32, BF16)], ids=str)
@pytest.mark.parametrize("counts,H,I", SHAPES, ids=ids)
def test_backward_on_random_values(counts, H, I, kind, dx_type, dw_type):
    b = Block(counts, H, I, 7 * H + I, False)
    a, e = b.kept(kind, False)
    dx = matrix(b.R, H, dx_type)
    dwgu, dwd = (torch.full(w.shape, NAN, device=DEV, dtype=dw_type) for w in (b.wgu, b.wd))
    ws = torch.empty(M.moe_ffn_backward_workspace_size(b.R, I), dtype=torch.uint8, device=DEV)
    M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx, dwgu, dwd, ws, act_exp=e)
    for k, s in b.experts():
        g, u = ref.act_values(a[s], e[s] if e is not None else None)
        want = ref.backward(b.dy[s], b.x[s], g, u, b.wgu[k], b.wd[k], dx_type, dw_type)
        near(dx[s], want["dx"], "dx")
        near(dwgu[k], want["dwgu"], "dw_gateup")
        near(dwd[k], want["dwd"], "dw_down")
    for k in range(b.E):
        if not counts[k]:
            assert bool((dwgu[k] == 0).all()) and bool((dwd[k] == 0).all())
    first = [t.clone() for t in (dx, dwgu, dwd)]
    M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx, dwgu, dwd, ws, act_exp=e)
    for t, u in zip(first, (dx, dwgu, dwd)):
        assert torch.equal(t.nan_to_num(), u.nan_to_num())  # the same bits again


def test_one_experts_nan_stays_with_it():
    """Neighbours share tiles and the last steps of a sum over rows."""
    counts, H, I = [5, 20, 70], 128, 64
    b = Block(counts, H, I, 11, False)
    a, e = b.kept("bf16", False)
    s = slice(b.o[1], b.o[2])
    ws = torch.empty(M.moe_ffn_backward_workspace_size(b.R, I), dtype=torch.uint8, device=DEV)

    def both():
        h, y = matrix(b.R, I, BF16), matrix(b.R, H, F32)
        dx, dwgu, dwd = matrix(b.R, H, F32), torch.empty_like(b.wgu), torch.empty_like(b.wd)
        M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y)
        M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx, dwgu, dwd, ws)
        return y, dx, dwgu, dwd

    clean = both()
    for bad in (NAN, float("inf")):
        b.x[s], b.dy[s], a[s] = bad, bad, bad
        b.wgu[1], b.wd[1] = bad, bad
        dirty = both()
        for k in (0, 2):
            r = slice(b.o[k], b.o[k + 1])
            assert torch.equal(clean[0][r], dirty[0][r]) and torch.equal(clean[1][r], dirty[1][r])
            assert torch.equal(clean[2][k], dirty[2][k]) and torch.equal(clean[3][k], dirty[3][k])
        assert not bool(torch.isfinite(dirty[0][s]).any()) and bool(dirty[2][1].isnan().any())


def test_a_wrong_row_is_seen_in_kept_values():
    """NaN and infinities of one row make its groups NaN, no others."""
    b = Block([3, 4], 64, 64, 13, False)
    b.x[4, 5] = NAN
    h, y = matrix(b.R, 64, BF16), matrix(b.R, 64, F32)
    q, e = keep("q8", b.R, 64)
    M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=q, act_exp=e)
    assert bool((e[4] == 255).all()) and bool((e[[0, 1, 2, 3, 5, 6]] != 255).all())


def test_nothing_to_do():
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    wgu, wd = torch.ones((2, 32, 8), dtype=BF16, device=DEV), torch.ones((2, 8, 16), dtype=BF16, device=DEV)
    none = lambda w, t=BF16: torch.empty((0, w), dtype=t, device=DEV)  # noqa: E731
    ws = torch.empty(0, dtype=torch.uint8, device=DEV)
    M.moe_ffn(none(8), wgu, wd, off, none(16), none(8), act=none(32))
    dwgu, dwd = torch.full_like(wgu, NAN), torch.full_like(wd, NAN)
    M.moe_ffn_backward(none(8), none(8), none(32), wgu, wd, off, none(8), dwgu, dwd, ws)
    assert bool((dwgu == 0).all()) and bool((dwd == 0).all())
    M.moe_ffn_backward(none(8), none(8), none(32), wgu, wd, off, none(8), dwgu.fill_(2), dwd, ws, accumulate=True)
    assert bool((dwgu == 2).all())


def test_offsets_are_clamped():
    """Offsets outside the rows or falling reach no row outside the buffers."""
    b = Block([10, 10], 64, 32, 17, False, behind=0)
    h, y = matrix(20, 32, BF16), matrix(20, 64, F32)
    ws = torch.empty(M.moe_ffn_backward_workspace_size(20, 32), dtype=torch.uint8, device=DEV)
    a, _ = b.kept("bf16", False)
    for o in ([-5, 10, 999], [20, 10, 0], [0, 1 << 30, -(1 << 30)]):
        off = torch.tensor(o, dtype=torch.int32, device=DEV)
        M.moe_ffn(b.x, b.wgu, b.wd, off, h, y)
        M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, off, y, torch.empty_like(b.wgu), torch.empty_like(b.wd), ws)
    torch.cuda.synchronize()
    off = torch.tensor([-5, 10, 999], dtype=torch.int32, device=DEV)
    M.moe_ffn(b.x, b.wgu, b.wd, off, h, y)
    want = matrix(20, 64, F32)
    M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, want)
    assert torch.equal(y, want)


def test_another_stream_and_a_graph():
    b = Block([40, 0, 90], 256, 128, 19, False)
    a, _ = keep("bf16", b.R, 128)
    h, y, dx = matrix(b.R, 128, BF16), matrix(b.R, 256, BF16), matrix(b.R, 256, BF16)
    dwgu, dwd = torch.empty_like(b.wgu), torch.empty_like(b.wd)
    ws = torch.empty(M.moe_ffn_backward_workspace_size(b.R, 128), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=a, stream=stream)
        M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx, dwgu, dwd, ws, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, dwgu, dwd)]

    def wipe():
        for t in (y, dx, dwgu, dwd, h, a):
            t.fill_(NAN)
        ws.fill_(255)

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(t.nan_to_num(), u.nan_to_num()) for t, u in zip(want, (y, dx, dwgu, dwd)))

    wipe()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        wipe()
        graph.replay()
        assert same()


def test_refusals_of_the_binding():
    b = Block([4], 64, 32, 23, False, behind=0)
    h, y, a = matrix(4, 32, BF16), matrix(4, 64, F32), matrix(4, 64, BF16)
    q, e = keep("q8", 4, 32)
    ws = torch.empty(M.moe_ffn_backward_workspace_size(4, 32), dtype=torch.uint8, device=DEV)
    dwgu, dwd = torch.empty_like(b.wgu), torch.empty_like(b.wd)
    bad = [
        lambda: M.moe_ffn(b.x.float(), b.wgu, b.wd, b.off, h, y),
        lambda: M.moe_ffn(b.x, b.wgu.float(), b.wd, b.off, h, y),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd[:, :, :24], b.off, h, y),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off.long(), h, y),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off[:1], h, y),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off, h[:3], y),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y[:3]),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=q),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=a, act_exp=e),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act_exp=e),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=q, act_exp=e[:, :1]),
        lambda: M.moe_ffn(b.x[:, :60], b.wgu[:, :, :60].contiguous(), b.wd[:, :60].contiguous(), b.off, h, y[:, :60]),
        lambda: M.moe_ffn(b.x.cpu(), b.wgu, b.wd, b.off, h, y),
        lambda: M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, b.x),
        lambda: M.moe_ffn_backward(b.dy, b.x, None, b.wgu, b.wd, b.off, None, dwgu, dwd, ws),
        lambda: M.moe_ffn_backward(b.dy, None, a, b.wgu, b.wd, b.off, None, dwgu, dwd, ws),
        lambda: M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, None, None, None, ws),
        lambda: M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, None, dwgu, dwd.float(), ws),
        lambda: M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, None, dwgu, dwd, ws[:-16]),
        lambda: M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, b.dy, dwgu, dwd, ws),
        lambda: M.moe_ffn_backward(b.dy, b.x, a, None, b.wd, b.off, y, None, dwd, ws),
        lambda: M.moe_ffn_backward(b.dy, b.x, q, b.wgu, b.wd, b.off, None, dwgu, dwd, ws),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(MoEError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_many_passes_with_few_rows():
    """Mostly experts without rows or with a few, many launches in a row: every wait ends and the bits stay."""
    E, H, I, T = 512, 256, 128, 160
    g = gen(29)
    ids = torch.randint(0, E, (T,), generator=g, device=DEV).sort().values
    off = torch.searchsorted(ids, torch.arange(E + 1, device=DEV)).to(torch.int32)
    x, dy = (torch.randn((T, H), generator=g, device=DEV).to(BF16) for _ in range(2))
    wgu, wd = (torch.randn(s, generator=g, device=DEV).to(BF16) / 16 for s in ((E, 2 * I, H), (E, H, I)))
    a, e = keep("q8", T, I)
    h, y, dx = matrix(T, I, BF16), matrix(T, H, BF16), matrix(T, H, BF16)
    dwgu, dwd = torch.empty_like(wgu), torch.empty_like(wd)
    ws = torch.empty(M.moe_ffn_backward_workspace_size(T, I), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = None
    for i in range(300):
        M.moe_ffn(x, wgu, wd, off, h, y, act=a, act_exp=e, dev_status=st)
        M.moe_ffn_backward(dy, x, a, wgu, wd, off, dx, dwgu, dwd, ws, act_exp=e, dev_status=st)
        if i % 50 == 0:
            assert int(st) == 0
            got = [t.clone() for t in (y, dx, dwgu, dwd)]
            want = want or got
            assert all(torch.equal(p, q) for p, q in zip(want, got))
    assert int(st) == 0


def test_gate_and_up_alone():
    """Without y: h and act, and no W_down is needed."""
    b = Block([5, 40], 128, 64, 31, False)
    h, y, a = matrix(b.R, 64, BF16), matrix(b.R, 128, F32), matrix(b.R, 128, BF16)
    M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=a)
    h2, a2 = matrix(b.R, 64, BF16), matrix(b.R, 128, BF16)
    M.moe_ffn(b.x, b.wgu, None, b.off, h2, None, act=a2)
    assert torch.equal(h.nan_to_num(), h2.nan_to_num()) and torch.equal(a.nan_to_num(), a2.nan_to_num())


def test_more_tiles_than_are_looked_up_ahead():
    """128 tiles of a pair are found at the start; here each has more."""
    H, I = 8, 8
    counts = [1_300_001, 0, 1_300_003]
    b = Block(counts, H, I, 37, True)
    h, y = matrix(b.R, I, BF16), matrix(b.R, H, F32)
    a, _ = b.kept("bf16", True)
    dx, dwgu, dwd = matrix(b.R, H, F32), torch.empty_like(b.wgu), torch.empty_like(b.wd, dtype=F32)
    ws = torch.empty(M.moe_ffn_backward_workspace_size(b.R, I), dtype=torch.uint8, device=DEV)
    M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y)
    M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx, None, dwd, ws)
    for k, s in b.experts():
        x, wgu, wd = b.x[s].double(), b.wgu[k].double(), b.wd[k].double()
        hh = ((x @ wgu[:I].t()).clamp_min(0) * (x @ wgu[I:].t())).to(BF16).double()
        assert torch.equal(y[s].double(), hh @ wd.t())
        g, u = a[s, :I].double(), a[s, I:].double()
        dh = b.dy[s].double() @ wd
        r = torch.where(g > 0, 1.0, 0.5)
        assert torch.equal(dx[s].double(), torch.cat([dh * u * r, dh * g * r], 1) @ wgu)
        want = b.dy[s].double().t() @ (g * r * u)
        assert float(want.abs().max()) < 2 ** 24
        assert torch.equal(dwd[k].double(), want)
    assert bool((dwd[1] == 0).all())


def test_two_streams_at_once():
    """Launches of two calls that share the GPU: each as if it were alone."""
    blocks = [Block([300, 0, 77, 500], 512, 256, s, False) for s in (41, 43)]
    runs = []
    for b in blocks:
        a, e = keep("q8", b.R, 256)
        o = [matrix(b.R, 256, BF16), matrix(b.R, 512, BF16), matrix(b.R, 512, BF16), torch.empty_like(b.wgu), torch.empty_like(b.wd)]
        ws = torch.empty(M.moe_ffn_backward_workspace_size(b.R, 256), dtype=torch.uint8, device=DEV)
        runs.append((b, a, e, o, ws))

    def go(r, stream=None):
        b, a, e, (h, y, dx, dwgu, dwd), ws = r
        M.moe_ffn(b.x, b.wgu, b.wd, b.off, h, y, act=a, act_exp=e, stream=stream)
        M.moe_ffn_backward(b.dy, b.x, a, b.wgu, b.wd, b.off, dx, dwgu, dwd, ws, act_exp=e, stream=stream)

    want = []
    for r in runs:
        go(r)
        torch.cuda.synchronize()
        want.append([t.clone() for t in r[3]])
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(20):
        for r, s in zip(runs, streams):
            go(r, s)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert all(torch.equal(t.nan_to_num(), v.nan_to_num()) for t, v in zip(r[3], w))


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("counts,H,I", [([[40, 0, 9, 300], [3, 200, 140, 6]], 256, 192),
                                        ([[2] * 48, [0, 4] * 24], 1024, 64), ([[1], [1]], 128, 2048)], ids=str)
def test_inputs_written_right_before(counts, H, I, graph):
    """Every input is overwritten by the launches just before a call, again and again: later launches of a call, which
    read offsets and weights before the one ahead of them has ended, see the call's own."""
    blocks = [Block(c, H, I, 61 + i, False) for i, c in enumerate(counts)]
    R, E = blocks[0].R, blocks[0].E
    assert all(b.R == R for b in blocks)
    now = Block(counts[0], H, I, 61, False)
    fields = ["x", "dy", "wgu", "wd", "off"]
    a, e = keep("q8", R, I)
    o = [torch.zeros(R, I, dtype=BF16, device=DEV), torch.zeros(R, H, dtype=BF16, device=DEV),
         torch.zeros(R, H, dtype=BF16, device=DEV), torch.zeros_like(now.wgu), torch.zeros_like(now.wd)]
    ws = torch.empty(M.moe_ffn_backward_workspace_size(R, I), dtype=torch.uint8, device=DEV)

    def step(b):
        for f in fields:
            getattr(now, f).copy_(getattr(b, f))
        for t in o:
            t.zero_()
        M.moe_ffn(now.x, now.wgu, now.wd, now.off, o[0], o[1], act=a, act_exp=e)
        for f in ("dy", "x", "wgu", "wd"):  # as written once more, the same values
            getattr(now, f).copy_(getattr(b, f))
        M.moe_ffn_backward(now.dy, now.x, a, now.wgu, now.wd, now.off, *o[2:], ws, act_exp=e)
        return [t.clone() for t in o]

    want = []
    for b in blocks:
        step(b)
        torch.cuda.synchronize()
        step(b)
        torch.cuda.synchronize()
        want.append([t.clone() for t in o])
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = [step(b) for _ in range(10) for b in blocks]
        for _ in range(5):
            g.replay()
    else:
        got = [step(b) for _ in range(50) for b in blocks]
    torch.cuda.synchronize()
    for i, t in enumerate(got):
        assert all(torch.equal(u.nan_to_num(), v.nan_to_num()) for u, v in zip(t, want[i % 2])), i
