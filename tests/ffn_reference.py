"""The experts' training operators in 64 bits, from their definitions, with error bounds.

As in block_reference.py a function returns (value, bound) pairs.  u = 2^-24 is
half a step of fp32.  The contractions' fp32 sums may drop bits instead of
rounding them, so a sum of n terms in any order is off by at most 2 n u
sum|terms|.  `half` of a type is half its step relative to the value (bf16
2^-8).  Bounds are first order with a factor 1.1 for the higher orders.
"""
import torch

from block_reference import F8, U, d, out

GROUP = 32
HALF = torch.finfo(torch.bfloat16).eps / 2


# ---------------------------------------------------------------- 8 bits
def _power(e):
    return ((e.to(torch.int64) + 1023) << 52).view(F8)


def quantise(x):
    """(q int8, exp uint8) of rows, exactly."""
    x = d(x)
    T, H = x.shape
    G = -(-H // GROUP)
    v = torch.nn.functional.pad(x, (0, G * GROUP - H)).view(T, G, GROUP)
    amax = v.abs().amax(2)
    bad = ~torch.isfinite(v).all(2)
    amax = torch.where(bad, torch.ones_like(amax), amax)
    m, p = torch.frexp(amax)  # amax = m 2^p, 1/2 <= m < 1
    e = torch.where(m <= 127 / 128, p - 7, p - 6).clamp(-126, 121)
    e = torch.where(amax == 0, torch.full_like(e, -126), e)
    q = torch.round(torch.nan_to_num(v) / _power(e)[..., None]).clamp(-127, 127)
    exp = torch.where(bad, torch.full_like(e, 255), e + 127)
    return q.view(T, G * GROUP)[:, :H].to(torch.int8), exp.to(torch.uint8)


def values(q, exp):
    """What 8-bit rows stand for, in 64 bits."""
    e = exp.to(torch.int64)
    s = torch.where(e == 255, torch.full(e.shape, float("nan"), dtype=F8, device=e.device), _power(e - 127))
    return d(q) * s.repeat_interleave(GROUP, 1)[:, :q.shape[1]]


def act_values(act, act_exp):
    """(g, u) of kept gate and up values."""
    I = act.shape[1] // 2
    if act_exp is None:
        return d(act[:, :I]), d(act[:, I:])
    G = act_exp.shape[1] // 2
    return values(act[:, :I], act_exp[:, :G]), values(act[:, I:], act_exp[:, G:])


# ---------------------------------------------------------------- the block
def dot(a, ab, b, bb):
    """a @ b of operands that are themselves off by ab and bb, with an fp32 sum."""
    n = a.shape[1]
    return a @ b, ab @ b.abs() + a.abs() @ bb + 2 * (n + 2) * U * (a.abs() @ b.abs())


def zeros(t):
    return torch.zeros_like(t)


def sigmoid(g):
    """r = 1 / (1 + exp(-g)) and how far it is off, relative: the fast exponential by 2 + 1.173 |g| units in the last
    place (2 u each), the sum by u, the fast quotient by 2 units."""
    return torch.sigmoid(g), (9 + 2.4 * g.abs()) * U


def forward(x, wgu, wd, dtype=torch.bfloat16):
    """One expert: {name: (value, bound)} of g, u (fp32), h and y."""
    x, wgu, wd = d(x), d(wgu), d(wd)
    I = wd.shape[1]
    a, ab = dot(x, zeros(x), wgu.t(), zeros(wgu.t()))
    g, u, gb, ub = a[:, :I], a[:, I:], ab[:, :I], ab[:, I:]
    sg, sb = sigmoid(g)
    h = g * sg * u
    # |silu'| <= 1.1; two products
    hb = 1.1 * u.abs() * gb + (g * sg).abs() * ub + gb * ub + (sb + 2 * U) * h.abs()
    h, hb = out(h, hb, torch.bfloat16)
    y, yb = dot(h, hb, wd.t(), zeros(wd.t()))
    return {"g": (g, gb), "u": (u, ub), "h": (h, hb), "y": out(y, yb, dtype)}


def backward(dy, x, g, u, wgu, wd, dx_type=torch.bfloat16, dw_type=torch.bfloat16):
    """One expert: {name: (value, bound)} of dx, dwgu and dwd from the kept g and u."""
    dy, wgu, wd = d(dy), d(wgu), d(wd)
    r, rb = sigmoid(g)
    dh, dhb = dot(dy, zeros(dy), wd, zeros(wd))
    sl = r * (1 + g * (1 - r))
    # r + g r - g r r: each term is at most r |g| or r, off by rb of r twice at most and four roundings
    slb = (2 * rb + 4 * U) * r * (1 + 2 * g.abs())
    dg = out(dh * u * sl, dhb * (u * sl).abs() + (dh * u).abs() * slb + 4 * U * (dh * u * sl).abs(), torch.bfloat16)
    du = out(dh * g * r, dhb * (g * r).abs() + (rb + 2 * U) * (dh * g * r).abs(), torch.bfloat16)
    h = out(g * r * u, (rb + 2 * U) * (g * r * u).abs(), torch.bfloat16)
    da, dab = torch.cat([dg[0], du[0]], 1), torch.cat([dg[1], du[1]], 1)
    got = {"dx": out(*dot(da, dab, wgu, zeros(wgu)), dx_type)}
    if x is not None:
        got["dwgu"] = out(*dot(da.t(), dab.t(), d(x), zeros(d(x))), dw_type)
    got["dwd"] = out(*dot(dy.t(), zeros(dy.t()), h[0], h[1]), dw_type)
    return got
