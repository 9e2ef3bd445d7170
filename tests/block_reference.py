"""The block operators in 64 bits, from their definitions, with error bounds.

Every function takes torch tensors of any type, computes in float64 and
returns {name: (value, bound)}: the exact value and how far fp32 arithmetic
with correctly rounded products and sums may be from it, element by element.
With u = 2^-24 (half a step of fp32), a sum of n terms computed in any order
is off by at most n u sum|terms|, a product of m factors by m u |product|;
`out` adds the rounding to the output's type (half a step: bf16 2^-8, relative).
The bounds are first order in u with a factor 1.1 for the higher orders and
2^-126 for results below fp32's normal range.
"""
import torch

U = 2.0 ** -24
F8 = torch.float64


def d(t):
    return t.to(F8)


def out(value, bound, dtype):
    half = torch.finfo(dtype).eps / 2
    bound = 1.1 * bound + 2.0 ** -126
    return value, bound + half * (value.abs() + bound)


def _rows(rows, inv):
    """rows[inv] with zeros for routes without a slot, and which have one."""
    kept = (inv >= 0) & (inv < rows.shape[0])
    if rows.shape[0] == 0:
        return torch.zeros(inv.shape + rows.shape[1:], dtype=F8, device=rows.device), kept
    v = d(rows)[torch.where(kept, inv, 0).long()]
    return torch.where(kept[..., None], v, torch.zeros((), dtype=F8, device=rows.device)), kept


def spread(tok, inv, w, into):
    """dispatch, and collect's gradient: the rows `into` after the call."""
    T, k = inv.shape
    kept = (inv >= 0) & (inv < into.shape[0])
    t, j = kept.nonzero(as_tuple=True)
    v = d(into).clone()
    wt = torch.ones((T, k), dtype=F8, device=inv.device) if w is None else d(w)
    v[inv[t, j].long()] = wt[t, j, None] * d(tok)[t]
    written = torch.zeros(into.shape[0], dtype=torch.bool, device=inv.device)
    written[inv[t, j].long()] = True
    val, bound = out(v, U * v.abs(), into.dtype)
    return val, torch.where(written[:, None], bound, torch.zeros((), dtype=F8, device=inv.device))


def join(rows, inv, w, add, dtype):
    """collect, and dispatch's gradient."""
    v, kept = _rows(rows, inv)
    if w is not None:
        v = v * torch.where(kept, d(w), torch.zeros((), dtype=F8, device=inv.device))[..., None]
    a = torch.zeros_like(v[:, 0]) if add is None else d(add)
    return out(a + v.sum(1), (inv.shape[1] + 2) * U * (a.abs() + v.abs().sum(1)), dtype)


def dots(rows, inv, tok):
    """dw of either gradient."""
    v, _ = _rows(rows, inv)
    p = v * d(tok)[:, None, :]
    return out(p.sum(-1), (p.shape[-1] + 1) * U * p.abs().sum(-1), torch.float32)


def rstd(x, eps):
    """1 / sqrt(mean x^2 + eps) and its relative bound: n roundings of the
    positive sum, the mean, eps, the root and the quotient."""
    r = 1.0 / (d(x).square().mean(1, keepdim=True) + eps).sqrt()
    return r, (x.shape[1] / 2 + 6) * U


def norm(x, y, gate, gamma_post, gamma_pre, scale, eps, post, x_type, y_type):
    """gate broadcasts against [T, H]."""
    got = {}
    sx = scale * d(x)
    z, zb = torch.zeros_like(sx), torch.zeros_like(sx)
    if y is not None:
        z, rel = d(y), 0.0
        if post:
            r, rel = rstd(d(y), eps)
            got["rstd_post"] = out(r[:, 0], rel * r[:, 0], torch.float32)
            z = z * r * (1.0 if gamma_post is None else 1.0 + d(gamma_post))
        if gate is not None:
            z = z * d(gate)
        zb = (rel + 8 * U) * z.abs()
    xo = sx + z
    xb = 3 * U * sx.abs() + zb + 2 * U * xo.abs()
    got["x_out"] = out(xo, xb, x_type)
    # the mean square moves by 2 mean|x dx|, the factor by half of that, relative
    r, rel = rstd(xo, eps)
    rel = rel + r * r * (xo.abs() * xb).mean(1, keepdim=True)
    got["rstd_pre"] = out(r[:, 0], (rel * r)[:, 0], torch.float32)
    gain = 1.0 if gamma_pre is None else 1.0 + d(gamma_pre)
    gabs = 1.0 if gamma_pre is None else gain.abs()
    n = xo * r * gain
    got["n_out"] = out(n, (rel + 6 * U) * n.abs() + xb * r * gabs, y_type)
    return got


def norm_grad(dx_out, dn, x_out, y, gate, gamma_post, gamma_pre, scale, r1, r2, post, x_type, y_type):
    """r1, r2: [T] as the forward call wrote them (inputs here)."""
    got = {}
    one = torch.ones((), dtype=F8, device=(dx_out if dx_out is not None else dn).device)
    base = dx_out if dx_out is not None else dn
    T, H = base.shape
    D = torch.zeros((T, H), dtype=F8, device=base.device) if dx_out is None else d(dx_out)
    Db = torch.zeros_like(D)
    if dn is not None:
        r = d(r2)[:, None]
        xh = d(x_out) * r
        g = one if gamma_pre is None else 1.0 + d(gamma_pre)
        u = d(dn) * g
        m, mabs = (u * xh).mean(1, keepdim=True), (u * xh).abs().mean(1, keepdim=True)
        D = D + r * (u - xh * m)
        Db = 5 * U * (D.abs() + r * (u.abs() + xh.abs() * mabs)) + r * xh.abs() * (H + 6) * U * mabs
        p = d(dn) * xh
        got["dgamma_pre"] = out(p.sum(0), (T + 4) * U * p.abs().sum(0), torch.float32)
    got["dx"] = out(scale * D, abs(scale) * (Db + U * D.abs()), x_type)
    if y is None:
        return got
    gt = one if gate is None else d(gate)
    g1 = one if gamma_post is None else 1.0 + d(gamma_post)
    rr = d(r1)[:, None] if post else one
    yh = d(y) * rr
    z = yh * g1
    a = D * gt * yh
    ab = (Db + 5 * U * D.abs()) * (gt * yh).abs()
    if post:
        v = D * gt * g1
        vb = (Db + 5 * U * D.abs()) * (gt * g1).abs()
        m, mabs = (v * yh).mean(1, keepdim=True), (v * yh).abs().mean(1, keepdim=True)
        mb = (vb * yh.abs()).mean(1, keepdim=True) + (H + 8) * U * mabs
        dy = rr * (v - yh * m)
        got["dy"] = out(dy, rr * (vb + yh.abs() * mb + 5 * U * (v.abs() + yh.abs() * mabs)), y_type)
        got["dgamma_post"] = out(a.sum(0), ab.sum(0) + (T + 6) * U * a.abs().sum(0), torch.float32)
    else:
        got["dy"] = out(D * gt, (Db + 3 * U * D.abs()) * gt.abs(), y_type)
    if gate is None:
        return got
    p = D * z
    pb = (Db + 6 * U * D.abs()) * z.abs()
    if gate.dim() == 1:
        got["dgate"] = out(p.sum(0), pb.sum(0) + (T + 6) * U * p.abs().sum(0), torch.float32)
    elif gate.shape[1] == 1 and gate.dtype != torch.bfloat16:  # bf16: a full gate of width 1
        s = p.sum(1, keepdim=True)
        got["dgate"] = out(s, pb.sum(1, keepdim=True) + (H + 6) * U * p.abs().sum(1, keepdim=True), torch.float32)
    else:
        got["dgate"] = out(p, pb, y_type)
    return got


def route_grad(dw, w, ids, x, w_router, add, dx_type):
    E, H = w_router.shape
    T, k = ids.shape
    dev = dw.device
    g, p = d(w) * d(dw), d(w)
    s, sabs = g.sum(1, keepdim=True), g.abs().sum(1, keepdim=True)
    dl = p * (d(dw) - s)
    dlb = p.abs() * ((k + 4) * U * (d(dw).abs() + sabs))
    got = {"dlogits": out(dl, dlb, torch.float32)}
    a = torch.zeros((T, H), dtype=F8, device=dev) if add is None else d(add)
    rows = d(w_router)[ids.long()]
    t = dl[..., None] * rows
    got["dx"] = out(a + t.sum(1), (dlb[..., None] * rows.abs()).sum(1) + (k + 2) * U * (a.abs() + t.abs().sum(1)),
                    dx_type)
    onto = torch.zeros((T, E), dtype=F8, device=dev)
    dense, denseb, absd = (onto.clone().scatter_add_(1, ids.long(), v) for v in (dl, dlb, dl.abs()))
    n = torch.bincount(ids.flatten().long(), minlength=E).to(F8)
    xa = d(x)
    got["dw_router"] = out(dense.t() @ xa, denseb.t() @ xa.abs() + (n + 2)[:, None] * U * (absd.t() @ xa.abs()),
                           torch.float32)
    got["dbias"] = out(dense.sum(0), denseb.sum(0) + (n + 2) * U * absd.sum(0), torch.float32)
    return got
