"""Cases of the block operators: tokens to experts and back, block norms, the router's gradient.

Each case is one call of one operator on data as a program holds it between
the layer's other calls.  With ``own`` the calls go to the package's entry
points; without it ``run`` computes the same outputs from elementary torch
operations in 32 bits.

A case names its operator (``op``) and

  T, H, k, E   tokens, row width, routes per token, experts
  rows         type of activation rows ("bf16" or "f32")
  stream       type of the residual stream's rows (norms), of dx (gradients)
  weights      whether the route weights are applied (dispatch)
  drop         share of the routes that have no slot (a full expert, padding)
  zipf         popularity of the experts: rank^-zipf; 0 is uniform
  gate         "none", "channel" [H], "token" [T,1] or "full" [T,H]
  post         whether the block's output is normalised before its gate
  pad          columns between the end of one row and the start of the next
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
SCALE = 0.75  # of the residual stream


def _case(name, op, T, H, k=10, E=512, rows="bf16", stream="f32", weights=True, drop=0.0, zipf=0.0, gate="none",
          post=True, pad=0):
    return {"name": name, "op": op, "T": T, "H": H, "k": k, "E": E, "rows": rows, "stream": stream,
            "weights": weights, "drop": drop, "zipf": zipf, "gate": gate, "post": post, "pad": pad}


def listed():
    return [
        # a decode block of 16 tokens brought into expert order
        _case("dispatch, decode", "dispatch", 16, 2560, weights=False, zipf=1.0),
        # a prompt of 4,096 tokens with the weights on the rows, some routes beyond their expert's capacity
        _case("dispatch, prompt, weighted", "dispatch", 4096, 2560, drop=0.05, zipf=0.5),
        # its gradient: the rows' sum per token and the gradient of the weights
        _case("dispatch gradient, prompt", "dispatch_bwd", 4096, 2560, drop=0.05, zipf=0.5, stream="bf16"),
        # fp32 expert outputs of a decode block, back in token order
        _case("collect, decode", "collect", 16, 2560, rows="f32", stream="bf16", zipf=1.0),
        # the largest training batch
        _case("collect gradient, batch", "collect_bwd", 16384, 2560, stream="bf16"),
        # a ragged one: odd width, few experts, fp32, padding tokens
        _case("collect gradient, ragged", "collect_bwd", 509, 1001, k=6, E=64, rows="f32", drop=0.1),
        # between two blocks while decoding one token
        _case("norm, one token", "norm", 1, 2560),
        # the same for a prompt, with a gate per channel
        _case("norm, prompt, gated", "norm", 4096, 2560, gate="channel"),
        # its gradient
        _case("norm gradient, prompt, gated", "norm_bwd", 4096, 2560, gate="channel"),
        # a bf16 stream with a gate per token, odd width
        _case("norm gradient, token gate", "norm_bwd", 8191, 1282, rows="bf16", stream="bf16", gate="token"),
        # the router of the small test layer
        _case("router gradient, small", "route_bwd", 16, 256, k=4, E=64),
        # the router of the whole layer on a prompt with popular experts
        _case("router gradient, prompt", "route_bwd", 4096, 2560, zipf=1.0),
    ]


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_bwd", "collect", "collect_bwd", "norm", "norm_bwd", "route_bwd"])

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    H = rng.choice([log(64, 8192), 8 * log(8, 1024), 128 * log(1, 64)])
    E = rng.choice([log(4, 1024), 64, 128, 512])
    k = min(E, log(1, 16))
    T = log(1, 16384)
    while T * k * H > 16384 * 10 * 2560 // 2 or T * H > 8192 * 2560:
        T = max(1, T // 2)
    rows, stream = rng.choice([("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
    return {"op": op, "T": T, "H": H, "k": k, "E": E, "rows": rows, "stream": stream,
            "weights": rng.random() < 0.7, "drop": rng.choice([0.0, 0.02, 0.3]), "zipf": rng.choice([0.0, 0.5, 1.0]),
            "gate": rng.choice(["none", "channel", "token", "full"]), "post": rng.random() < 0.8,
            "pad": rng.choice([0, 0, 8, 3])}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T, H, k, E, pad = case["T"], case["H"], case["k"], case["E"], case["pad"]
    R = T * k
    rows, stream = TYPES[case["rows"]], TYPES[case["stream"]]
    op = case["op"]

    def normal(n, dtype, std=1.0):
        """n rows of H columns, `pad` columns apart in memory."""
        v = torch.randn((n, H + pad), generator=g, device="cuda") * std
        return v.to(dtype)[:, :H]

    def empty(n, dtype):
        return torch.zeros((n, H + pad), device="cuda", dtype=dtype)[:, :H]

    s = {"case": dict(case)}
    if op.startswith("norm"):
        s["x"] = normal(T, stream)
        s["y"] = normal(T, rows, 0.5)
        s["gamma_post"] = torch.randn(H, generator=g, device="cuda") * 0.1 if case["post"] else None
        s["gamma_pre"] = torch.randn(H, generator=g, device="cuda") * 0.1
        gate = case["gate"]
        s["gate"] = {"none": lambda: None,
                     "channel": lambda: torch.rand(H, generator=g, device="cuda"),
                     "token": lambda: torch.rand((T, 1), generator=g, device="cuda"),
                     "full": lambda: normal(T, rows)}[gate]()
        if op == "norm":
            s["x_out"], s["n_out"] = empty(T, stream), empty(T, rows)
            s["rstd_post"], s["rstd_pre"] = (torch.zeros(T, device="cuda") for _ in range(2))
            return s
        # what the forward pass left: its stream and the two norms' factors
        y = s["y"].float()
        s["rstd_post"] = torch.rsqrt((y * y).mean(-1) + EPS) if case["post"] else torch.ones(T, device="cuda")
        s["x_out"] = s.pop("x")
        xo = s["x_out"].float()
        s["rstd_pre"] = torch.rsqrt((xo * xo).mean(-1) + EPS)
        s["dx_out"], s["dn"] = normal(T, stream), normal(T, rows)
        s["dx"], s["dy"] = empty(T, stream), empty(T, rows)
        s["dgamma_post"] = torch.zeros(H, device="cuda") if case["post"] else None
        s["dgamma_pre"] = torch.zeros(H, device="cuda")
        s["dgate"] = {"none": lambda: None, "channel": lambda: torch.zeros(H, device="cuda"),
                      "token": lambda: torch.zeros((T, 1), device="cuda"), "full": lambda: empty(T, rows)}[gate]()
        return s

    # routes as the router and the grouping leave them: k distinct experts a
    # token, renormalised weights, slots in expert order, stable
    pop = -case["zipf"] * torch.log(torch.randperm(E, generator=g, device="cuda").float() + 1)
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_min(1e-20)
    score = pop - torch.log((-torch.log(noise)).clamp_min(1e-20))  # Gumbel noise: draws without replacement
    top, ids = score.topk(k, dim=1)
    s["w"] = torch.softmax(top, dim=1).contiguous()
    s["ids"] = ids.to(torch.int32).contiguous()
    key, order = s["ids"].view(-1).sort(stable=True)
    s["perm"] = order.to(torch.int32)
    inv = torch.empty(R, device="cuda", dtype=torch.int32)
    inv[order] = torch.arange(R, device="cuda", dtype=torch.int32)
    inv = inv.view(T, k)
    edge = torch.arange(E + 1, device="cuda", dtype=torch.int32)
    s["offsets"] = torch.searchsorted(key.contiguous(), edge).to(torch.int32)
    if case["drop"] > 0:
        gone = torch.rand((T, k), generator=g, device="cuda") < case["drop"]
        gone[T - T // 32:] = True  # padding behind the last sequence
        inv = torch.where(gone, torch.full_like(inv, -1), inv)
    s["inv"] = inv.contiguous()
    if op == "dispatch":
        s["x"], s["x_perm"] = normal(T, rows), empty(R, rows)
    elif op == "dispatch_bwd":
        s["dx_perm"], s["x"] = normal(R, rows), normal(T, rows)
        s["dx"], s["add"] = empty(T, stream), normal(T, stream)
        s["dw"] = torch.zeros((T, k), device="cuda")
    elif op == "collect":
        s["y_perm"], s["out"] = normal(R, rows), empty(T, stream)
    elif op == "collect_bwd":
        s["y_perm"], s["dout"], s["dy_perm"] = normal(R, rows), normal(T, stream), empty(R, rows)
        s["dw"] = torch.zeros((T, k), device="cuda")
    elif op == "route_bwd":
        s["x"], s["w_router"] = normal(T, torch.bfloat16), normal(E, torch.bfloat16, 0.02)
        s["dw"] = torch.randn((T, k), generator=g, device="cuda")
        s["dlogits"] = torch.zeros((T, k), device="cuda")
        s["dx"], s["add"] = empty(T, stream), normal(T, stream)
        s["dw_router"], s["dbias"] = empty(E, torch.float32), torch.zeros(E, device="cuda")
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import sparse_moe_routed_gb300 as M

    c = s["case"]
    op = c["op"]
    w = s.get("w") if c["weights"] else None
    if op == "dispatch":
        M.moe_dispatch(s["x"], s["inv"], s["x_perm"], w=w)
        return {"x_perm": s["x_perm"]}
    if op == "dispatch_bwd":
        if w is None:
            M.moe_dispatch_backward(s["dx_perm"], s["inv"], s["dx"], add=s["add"])
            return {"dx": s["dx"]}
        M.moe_dispatch_backward(s["dx_perm"], s["inv"], s["dx"], w=w, x=s["x"], dw=s["dw"], add=s["add"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "collect":
        M.moe_collect(s["y_perm"], s["inv"], s["w"], s["out"])
        return {"out": s["out"]}
    if op == "collect_bwd":
        M.moe_collect_backward(s["dout"], s["y_perm"], s["inv"], s["w"], s["dy_perm"], s["dw"])
        return {"dy_perm": s["dy_perm"], "dw": s["dw"]}
    if op == "norm":
        M.moe_block_norm(s["x"], s["y"], s["x_out"], s["n_out"], gamma_post=s["gamma_post"],
                         gamma_pre=s["gamma_pre"], gate=s["gate"], scale=SCALE, eps=EPS, post_norm=c["post"],
                         rstd_post=s["rstd_post"] if c["post"] else None, rstd_pre=s["rstd_pre"])
        return {k: s[k] for k in ("x_out", "n_out", "rstd_pre") + (("rstd_post",) if c["post"] else ())}
    if op == "norm_bwd":
        if "ws" not in s:
            s["ws"] = torch.empty(M.moe_block_norm_workspace_size(c["T"], c["H"]), dtype=torch.uint8, device="cuda")
        M.moe_block_norm_backward(s["dx_out"], s["dn"], s["x_out"], s["y"], s["dx"], s["dy"], s["ws"],
                                  gamma_post=s["gamma_post"], gamma_pre=s["gamma_pre"], gate=s["gate"], scale=SCALE,
                                  post_norm=c["post"], rstd_post=s["rstd_post"] if c["post"] else None,
                                  rstd_pre=s["rstd_pre"], dgate=s["dgate"], dgamma_post=s["dgamma_post"],
                                  dgamma_pre=s["dgamma_pre"])
        return {k: s[k] for k in ("dx", "dy", "dgate", "dgamma_post", "dgamma_pre") if s[k] is not None}
    if "ws" not in s:
        s["ws"] = torch.empty(M.moe_route_backward_workspace_size(c["T"], c["k"], c["E"], c["H"]), dtype=torch.uint8,
                              device="cuda")
    M.moe_route_backward(s["dw"], s["w"], s["ids"], s["x"], s["w_router"], s["offsets"], s["perm"], s["dlogits"],
                         s["dx"], s["dw_router"], s["dbias"], s["ws"], add=s["add"])
    return {k: s[k] for k in ("dlogits", "dx", "dw_router", "dbias")}


def _plain(s):
    c = s["case"]
    op, T, k, E = c["op"], c["T"], c["k"], c["E"]
    rows, stream = TYPES[c["rows"]], TYPES[c["stream"]]
    if op.startswith("norm"):
        return _plain_norm(s, c, rows, stream)
    if op == "route_bwd":
        w, dw = s["w"], s["dw"]
        dl = w * (dw - (w * dw).sum(-1, keepdim=True))
        dense = torch.zeros((T, E), device=dl.device).scatter(1, s["ids"].long(), dl)
        dx = s["add"].float() + dense @ s["w_router"].float()
        return {"dlogits": dl, "dx": dx.to(stream), "dw_router": dense.t() @ s["x"].float(), "dbias": dense.sum(0)}
    inv, perm = s["inv"].long(), s["perm"].long()
    kept = inv >= 0
    if op in ("dispatch", "collect_bwd"):
        # per slot: its token's row, times its route's weight
        src = s["x"] if op == "dispatch" else s["dout"]
        out = s["x_perm"] if op == "dispatch" else s["dy_perm"]
        v = src.float()[perm // k]
        if c["weights"] or op == "collect_bwd":
            v = v * s["w"].view(-1)[perm][:, None]
        v = torch.where(kept.view(-1)[perm][:, None], v.to(rows), out)
        if op == "dispatch":
            return {"x_perm": v}
        dot = (s["dout"].float()[:, None, :] * s["y_perm"].float()[inv.clamp_min(0)]).sum(-1)
        return {"dy_perm": v, "dw": torch.where(kept, dot, torch.zeros_like(dot))}
    # per token: its routes' rows, times their weights
    src = s["dx_perm"] if op == "dispatch_bwd" else s["y_perm"]
    v = torch.where(kept[:, :, None], src.float()[inv.clamp_min(0)], torch.zeros((), device=src.device))
    use_w = op == "collect" or c["weights"]
    total = (v * s["w"][:, :, None] if use_w else v).sum(1)
    if op == "collect":
        return {"out": total.to(stream)}
    dx = (total + s["add"].float()).to(stream)
    if not use_w:
        return {"dx": dx}
    return {"dx": dx, "dw": (v * s["x"].float()[:, None, :]).sum(-1)}


def _plain_norm(s, c, rows, stream):
    y = s["y"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    gpost = 1.0 + s["gamma_post"] if c["post"] else 1.0
    gpre = 1.0 + s["gamma_pre"]
    if c["op"] == "norm":
        z = y
        out = {}
        if c["post"]:
            r1 = torch.rsqrt((y * y).mean(-1) + EPS)
            out["rstd_post"] = r1
            z = y * r1[:, None] * gpost
        xo = SCALE * s["x"].float() + gate * z
        r2 = torch.rsqrt((xo * xo).mean(-1) + EPS)
        out.update(x_out=xo.to(stream), n_out=(xo * r2[:, None] * gpre).to(rows), rstd_pre=r2)
        return out
    xo, dn, r2 = s["x_out"].float(), s["dn"].float(), s["rstd_pre"][:, None]
    u = dn * gpre
    d = s["dx_out"].float() + r2 * u - xo * r2 * r2 * r2 * (u * xo).mean(-1, keepdim=True)
    out = {"dx": (SCALE * d).to(stream), "dgamma_pre": (dn * xo * r2).sum(0)}
    dz = d * gate
    if c["post"]:
        r1 = s["rstd_post"][:, None]
        z = y * r1 * gpost
        v = dz * gpost
        out["dy"] = (r1 * v - y * r1 * r1 * r1 * (v * y).mean(-1, keepdim=True)).to(rows)
        out["dgamma_post"] = (dz * y * r1).sum(0)
    else:
        z = y
        out["dy"] = dz.to(rows)
    if c["gate"] == "channel":
        out["dgate"] = (d * z).sum(0)
    elif c["gate"] == "token":
        out["dgate"] = (d * z).sum(-1, keepdim=True)
    elif c["gate"] == "full":
        out["dgate"] = (d * z).to(rows)
    return out



def work(case):
    c = case
    T, H, k, E = c["T"], c["H"], c["k"], c["E"]
    a = 2 if c["rows"] == "bf16" else 4
    r = 2 if c["stream"] == "bf16" else 4
    kept = T * k * (1.0 - c["drop"])
    op = c["op"]
    wts = c["weights"] or op.startswith("collect")
    index = T * k * (8 if wts else 4)
    if op == "dispatch":
        return {"bytes": T * H * a + kept * H * a + index, "flops": kept * H}
    if op == "dispatch_bwd":
        return {"bytes": kept * H * a + (T * H * a + T * k * 4 if c["weights"] else 0) + 2 * T * H * r + index,
                "flops": kept * H * (4 if c["weights"] else 1)}
    if op == "collect":
        return {"bytes": kept * H * a + T * H * r + index, "flops": 2 * kept * H}
    if op == "collect_bwd":
        return {"bytes": T * H * r + 2 * kept * H * a + index + T * k * 4, "flops": 3 * kept * H}
    if op.startswith("norm"):
        vec = H * 4 * (1 + (1 if c["post"] else 0) + (1 if c["gate"] == "channel" else 0))
        vec += T * 4 if c["gate"] == "token" else T * H * a if c["gate"] == "full" else 0
        if op == "norm":
            return {"bytes": 2 * T * H * (a + r) + vec + 8 * T, "flops": 10 * T * H}
        return {"bytes": 3 * T * H * (a + r) + 2 * vec + 8 * T, "flops": 24 * T * H}
    return {"bytes": T * H * 2 + E * H * 2 + 2 * T * H * r + E * H * 4 + T * k * 20 + E * 8, "flops": 4 * T * k * H}


def exact(case, seed):
    """The definitions, route by route or row by row, in 64 bits."""
    s = prepare(case, seed)
    c, op = case, case["op"]
    T, H, k, E = c["T"], c["H"], c["k"], c["E"]
    f8 = torch.float64
    if op == "norm":
        return _exact_norm(s, c)
    if op == "norm_bwd":
        return _exact_norm_bwd(s, c)
    w = s["w"].to(f8)
    if op == "route_bwd":
        g = s["dw"].to(f8)
        # the Jacobian of the softmax over a token's k logits, written out
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        dl = torch.einsum("tij,tj->ti", jac, g)
        dx, dwr = s["add"].to(f8).clone(), torch.zeros((E, H), device="cuda", dtype=f8)
        for j in range(k):
            e = s["ids"][:, j].long()
            dx += dl[:, j, None] * s["w_router"].to(f8)[e]
            dwr.index_add_(0, e, dl[:, j, None] * s["x"].to(f8))
        db = torch.zeros(E, device="cuda", dtype=f8).index_add_(0, s["ids"].view(-1).long(), dl.view(-1))
        return {"dlogits": dl, "dx": dx, "dw_router": dwr, "dbias": db}
    one = c["weights"] or op.startswith("collect")
    if op == "dispatch":
        out = torch.zeros((T * k, H), device="cuda", dtype=f8)
    elif op == "collect_bwd":
        out, dw = torch.zeros((T * k, H), device="cuda", dtype=f8), torch.zeros((T, k), device="cuda", dtype=f8)
    elif op == "collect":
        out = torch.zeros((T, H), device="cuda", dtype=f8)
    else:
        out, dw = s["add"].to(f8).clone(), torch.zeros((T, k), device="cuda", dtype=f8)
    for j in range(k):
        t = (s["inv"][:, j] >= 0).nonzero().view(-1)
        at = s["inv"][t, j].long()
        wj = w[t, j, None] if one else 1.0
        if op == "dispatch":
            out[at] = wj * s["x"][t].to(f8)
        elif op == "collect":
            out[t] += wj * s["y_perm"][at].to(f8)
        elif op == "collect_bwd":
            d = s["dout"][t].to(f8)
            out[at] = wj * d
            dw[t, j] = (d * s["y_perm"][at].to(f8)).sum(1)
        else:
            d = s["dx_perm"][at].to(f8)
            out[t] += wj * d
            dw[t, j] = (d * s["x"][t].to(f8)).sum(1)
    if op == "dispatch":
        return {"x_perm": out}
    if op == "collect":
        return {"out": out}
    if op == "collect_bwd":
        return {"dy_perm": out, "dw": dw}
    return {"dx": out, "dw": dw} if c["weights"] else {"dx": out}


def _exact_norm(s, c):
    f8 = torch.float64
    y = s["y"].to(f8)
    z, got = y, {}
    if c["post"]:
        got["rstd_post"] = 1.0 / (y.square().mean(1) + EPS).sqrt()
        z = y * got["rstd_post"][:, None] * (1.0 + s["gamma_post"].to(f8))
    if s["gate"] is not None:
        z = z * s["gate"].to(f8)
    xo = s["x"].to(f8) * SCALE + z
    got["rstd_pre"] = 1.0 / (xo.square().mean(1) + EPS).sqrt()
    got["x_out"] = xo
    got["n_out"] = xo * got["rstd_pre"][:, None] * (1.0 + s["gamma_pre"].to(f8))
    return got


def _exact_norm_bwd(s, c):
    f8 = torch.float64
    xo, y, dn = s["x_out"].to(f8), s["y"].to(f8), s["dn"].to(f8)
    H = xo.shape[1]
    xhat = xo * s["rstd_pre"].to(f8)[:, None]  # the normalised stream
    u = dn * (1.0 + s["gamma_pre"].to(f8))
    d = s["dx_out"].to(f8) + s["rstd_pre"].to(f8)[:, None] * (u - xhat * ((u * xhat).sum(1, keepdim=True) / H))
    got = {"dx": d * SCALE, "dgamma_pre": (dn * xhat).sum(0)}
    gate = s["gate"].to(f8) if s["gate"] is not None else torch.ones((), dtype=f8, device=xo.device)
    if c["post"]:
        r1 = s["rstd_post"].to(f8)[:, None]
        gain = 1.0 + s["gamma_post"].to(f8)
        yhat = y * r1
        v = d * gate * gain
        got["dy"] = r1 * (v - yhat * ((v * yhat).sum(1, keepdim=True) / H))
        got["dgamma_post"] = (d * gate * yhat).sum(0)
        z = yhat * gain
    else:
        got["dy"], z = d * gate, y
    if c["gate"] == "channel":
        got["dgate"] = (d * z).sum(0)
    elif c["gate"] == "token":
        got["dgate"] = (d * z).sum(1, keepdim=True)
    elif c["gate"] == "full":
        got["dgate"] = d * z
    return got
