"""Cases of the experts' training operators: the gated feed-forward block with its backward pass, and
activation checkpoints in 8 bits with their use in that pass.

Each case is one pass on data as a program holds it.  With ``own`` the calls go to the package's entry
points; without it ``run`` computes the same outputs from elementary torch operations in 32 bits.

A case names its operator (``op``):

  checkpoint   rows of activations into 8 bits, and back
  restore      8-bit token rows back into bf16 rows in expert order
  ffn          the block's forward pass, which keeps the gate and up values
  ffn_bwd      its backward pass from kept values
  step         both, with the tokens and the gate and up values kept in 8 bits between them

and T, k, E, H, I (tokens, routes per token, experts, row width, intermediate width), ``rows`` (type of
checkpointed rows), ``act`` (how gate and up values are kept: "bf16" or "q8"), ``zipf`` (popularity of the
experts: rank^-zipf), ``drop`` (share of the routes without a slot) and ``pad`` (columns between the end of
one checkpointed row and the start of the next).

8 bits: 32 columns of a row share the smallest power of two 2^e, -126 <= e <= 121, with max|x| <= 127 * 2^e;
a value is the whole number next to x / 2^e (ties to even, at most 127 either way) times 2^e.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32


def _case(name, op, T, H, k=1, E=1, I=0, rows="bf16", act="bf16", zipf=0.0, drop=0.0, pad=0):
    return {"name": name, "op": op, "T": T, "H": H, "k": k, "E": E, "I": I, "rows": rows, "act": act, "zipf": zipf,
            "drop": drop, "pad": pad}


def listed():
    return [
        # a decode block's residual stream kept for later
        _case("checkpoint, decode block", "checkpoint", 16, 2560),
        # odd width and stride
        _case("checkpoint, ragged", "checkpoint", 509, 1001, pad=3),
        # the fp32 residual stream of the largest training batch
        _case("checkpoint, batch, fp32", "checkpoint", 16384, 2560, rows="f32"),
        # token rows of a prompt-sized batch back in expert order, for the weight gradients
        _case("restore, prompt", "restore", 4096, 2560, k=10, E=512, drop=0.05),
        # the small test layer
        _case("ffn, tiny", "ffn", 16, 256, k=4, E=64, I=64),
        # the whole layer on a prompt-sized batch
        _case("ffn, prompt", "ffn", 4096, 2560, k=10, E=512, I=640),
        # one dense block, as a shared expert is
        _case("ffn, dense", "ffn", 8192, 4096, I=8192),
        # few popular experts, padding tokens, sizes off every tile
        _case("ffn gradient, ragged", "ffn_bwd", 509, 1000, k=6, E=64, I=200, zipf=0.5, drop=0.1, act="q8"),
        # the largest training batch of the whole layer
        _case("ffn gradient, batch", "ffn_bwd", 16384, 2560, k=10, E=512, I=640),
        # the dense block's gradient
        _case("ffn gradient, dense", "ffn_bwd", 8192, 4096, I=8192, act="q8"),
        # a training step of the small test layer's experts
        _case("step, tiny", "step", 16, 256, k=4, E=64, I=64, act="q8"),
        # a training step of the whole layer's experts on a prompt-sized batch
        _case("step, prompt", "step", 4096, 2560, k=10, E=512, I=640, act="q8"),
    ]


def draw(rng):
    op = rng.choice(["checkpoint", "restore", "ffn", "ffn", "ffn_bwd", "ffn_bwd", "step", "step"])

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    T = log(1, 16384)
    if op == "checkpoint":
        H = rng.choice([log(1, 8192), 128 * log(1, 64)])
        while T * H > 16384 * 2560:
            T = max(1, T // 2)
        return {"op": op, "T": T, "H": H, "k": 1, "E": 1, "I": 0, "rows": rng.choice(["bf16", "f32"]), "act": "bf16",
                "zipf": 0.0, "drop": 0.0, "pad": rng.choice([0, 0, 8, 3])}
    E = rng.choice([1, log(2, 512), 64, 512])
    k = min(E, log(1, 16))
    zipf = rng.choice([0.0, 0.0, 0.5])
    if op == "restore":
        H, I = rng.choice([log(64, 8192), 128 * log(1, 64)]), 0
        while T * k * H > 4096 * 10 * 2560:
            T = max(1, T // 2)
    else:
        H = rng.choice([8 * log(8, 640), 128 * log(1, 40)])
        I = rng.choice([8 * log(4, 640), 64 * log(1, 80)])
        while E * H * I > 512 * 2560 * 640:
            E = max(1, E // 2)
        k = min(E, k)
        # no more work than the dense block's, no more rows than the largest batch
        while T * k * H * I > 8192 * 4096 * 8192 // 2 or T * k * max(H, 2 * I) > 16384 * 10 * 2560 // 2:
            T = max(1, T // 2)
        if T * E > 4096 * 64:  # the most popular expert's rows times the experts stay within reach
            zipf = 0.0
    return {"op": op, "T": T, "H": H, "k": k, "E": E, "I": I, "rows": "bf16", "act": rng.choice(["bf16", "q8"]),
            "zipf": zipf, "drop": rng.choice([0.0, 0.0, 0.1]) if T >= 32 else 0.0, "pad": 0}


# ---------------------------------------------------------------- inputs
def _power(e):
    """2^e in 32 bits, exactly: a power function may be off in the last bit."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _to_8_bits(x):
    """(whole numbers, exponents + 127) of rows of any width, group by group."""
    T, H = x.shape
    G = -(-H // GROUP)
    v = torch.nn.functional.pad(x.float(), (0, G * GROUP - H)).view(T, G, GROUP)
    m, p = torch.frexp(v.abs().amax(-1))  # amax = m * 2^p, 0.5 <= m < 1
    e = torch.where(m <= 127 / 128, p - 7, p - 6).clamp(-126, 121)
    q = (v * _power(-e)[:, :, None]).round().clamp(-127, 127)
    return q.view(T, G * GROUP)[:, :H].to(torch.int8), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, T, H, k, E, I, pad = (case[n] for n in ("op", "T", "H", "k", "E", "I", "pad"))
    bf = torch.bfloat16

    def normal(n, w, std=1.0, dtype=bf):
        return torch.randn((n, w), generator=g, device="cuda", dtype=dtype) * std

    s = {"case": dict(case)}
    if op == "checkpoint":
        rows = TYPES[case["rows"]]
        # activations: channels of different size, a few large ones
        size = torch.exp(torch.randn(H, generator=g, device="cuda"))
        x = torch.randn((T, H), generator=g, device="cuda") * size
        s["x"] = torch.zeros((T, H + pad), device="cuda", dtype=rows)[:, :H]
        s["x"].copy_(x)
        s["q"] = torch.zeros((T, H), device="cuda", dtype=torch.int8)
        s["exp"] = torch.zeros((T, -(-H // GROUP)), device="cuda", dtype=torch.uint8)
        s["out"] = torch.zeros((T, H + pad), device="cuda", dtype=rows)[:, :H]
        return s

    # routes as the router and the grouping leave them: k distinct experts a
    # token, slots in expert order, the kept ones first
    pop = -case["zipf"] * torch.log(torch.randperm(E, generator=g, device="cuda").float() + 1)
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_min(1e-20)
    ids = (pop - torch.log((-torch.log(noise)).clamp_min(1e-20))).topk(k, dim=1).indices.view(-1)
    if case["drop"] > 0:
        gone = torch.rand(T * k, generator=g, device="cuda") < case["drop"]
        gone[(T - T // 32) * k:] = True  # padding behind the last sequence
        ids = torch.where(gone, torch.full_like(ids, E), ids)
    key, order = ids.sort(stable=True)
    R = T * k
    inv = torch.empty(T * k, device="cuda", dtype=torch.int32)
    inv[order] = torch.arange(T * k, device="cuda", dtype=torch.int32)
    s["inv"] = torch.where(ids < E, inv, torch.full_like(inv, -1)).view(T, k)
    s["token"] = order // k  # of each slot
    s["expert"] = key.contiguous()  # of each slot; E behind the last expert's rows, which no call writes
    edge = torch.arange(E + 1, device="cuda")
    s["offsets"] = torch.searchsorted(key, edge).to(torch.int32)
    s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))
    if op == "restore":
        s["q"], s["exp"] = _to_8_bits(normal(T, H))
        s["x_perm"] = torch.zeros((R, H), device="cuda", dtype=bf)
        return s

    s["w_gateup"] = normal(E * 2 * I, H, 1.0 / math.sqrt(H)).view(E, 2 * I, H)
    s["w_down"] = normal(E * H, I, 1.0 / math.sqrt(I)).view(E, H, I)
    s["h"] = torch.zeros((R, I), device="cuda", dtype=bf)
    if op in ("ffn", "step"):
        x = normal(T, H)
        s["y"] = torch.zeros((R, H), device="cuda", dtype=bf)
        s["x_perm"] = x[s["token"]] if op == "ffn" else torch.zeros((R, H), device="cuda", dtype=bf)
        if op == "step":
            s["x"] = x
            s["q"] = torch.zeros((T, H), device="cuda", dtype=torch.int8)
            s["exp"] = torch.zeros((T, -(-H // GROUP)), device="cuda", dtype=torch.uint8)
        if case["act"] == "q8":
            s["act"] = torch.zeros((R, 2 * I), device="cuda", dtype=torch.int8)
            s["act_exp"] = torch.zeros((R, 2 * (-(-I // GROUP))), device="cuda", dtype=torch.uint8)
        else:
            s["act"], s["act_exp"] = torch.zeros((R, 2 * I), device="cuda", dtype=bf), None
    if op in ("ffn_bwd", "step"):
        s["dy"] = normal(R, H)
        if op == "ffn_bwd":
            s["x_perm"], s["act"], s["act_exp"] = normal(R, H), normal(R, 2 * I), None
            if case["act"] == "q8":
                (qg, eg), (qu, eu) = _to_8_bits(s["act"][:, :I]), _to_8_bits(s["act"][:, I:])
                s["act"], s["act_exp"] = torch.cat([qg, qu], 1), torch.cat([eg, eu], 1)
        s["dx"] = torch.zeros((R, H), device="cuda", dtype=bf)
        s["dw_gateup"], s["dw_down"] = torch.zeros_like(s["w_gateup"]), torch.zeros_like(s["w_down"])
    return s


# ---------------------------------------------------------------- a pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import sparse_moe_routed_gb300 as M

    op = s["case"]["op"]
    if op == "checkpoint":
        M.moe_checkpoint_save(s["x"], s["q"], s["exp"])
        M.moe_checkpoint_load(s["q"], s["exp"], s["out"])
        return {"out": s["out"]}
    if op == "restore":
        M.moe_checkpoint_load(s["q"], s["exp"], s["x_perm"], inv_perm=s["inv"])
        return {"x_perm": s["x_perm"]}
    out = {}
    if op == "step":
        M.moe_checkpoint_save(s["x"], s["q"], s["exp"])
        M.moe_dispatch(s["x"], s["inv"], s["x_perm"])
    if op in ("ffn", "step"):
        M.moe_ffn(s["x_perm"], s["w_gateup"], s["w_down"], s["offsets"], s["h"], s["y"], act=s["act"],
                  act_exp=s["act_exp"])
        out["y"] = s["y"]
        if op == "ffn":
            if s["case"]["act"] == "q8":  # the values that the 8 bits stand for, gate and up
                I, G = s["case"]["I"], s["act_exp"].shape[1] // 2
                if "values" not in s:
                    s["values"] = torch.empty(s["act"].shape, dtype=torch.bfloat16, device="cuda")
                M.moe_checkpoint_load(s["act"][:, :I], s["act_exp"][:, :G], s["values"][:, :I])
                M.moe_checkpoint_load(s["act"][:, I:], s["act_exp"][:, G:], s["values"][:, I:])
                out["act"] = s["values"]
            else:
                out["act"] = s["act"]
            return out
        M.moe_checkpoint_load(s["q"], s["exp"], s["x_perm"], inv_perm=s["inv"])
    if "ws" not in s:
        s["ws"] = torch.empty(M.moe_ffn_backward_workspace_size(len(s["dy"]), s["case"]["I"]), dtype=torch.uint8,
                              device="cuda")
    M.moe_ffn_backward(s["dy"], s["x_perm"], s["act"], s["w_gateup"], s["w_down"], s["offsets"], s["dx"],
                       s["dw_gateup"], s["dw_down"], s["ws"], act_exp=s["act_exp"])
    out.update(dx=s["dx"], dw_gateup=s["dw_gateup"], dw_down=s["dw_down"])
    return out


def _values(q, exp):
    """What 8-bit rows stand for."""
    scale = _power(exp.to(torch.int32) - 127).repeat_interleave(GROUP, 1)[:, :q.shape[1]]
    return q.float() * scale


def _through_8_bits(x):
    return _values(*_to_8_bits(x))


def _plain(s):
    c = s["case"]
    op, E, I = c["op"], c["E"], c["I"]
    if op == "checkpoint":
        return {"out": _through_8_bits(s["x"]).to(s["x"].dtype)}
    if op == "restore":
        x = _values(s["q"], s["exp"])[s["token"]].to(torch.bfloat16)
        return {"x_perm": torch.where(s["expert"][:, None] < E, x, s["x_perm"])}

    # slots in a table of E experts by the most rows that one has: one batched product for all; the rows
    # behind the last expert's share one place after it
    off, most, bf = s["offsets"].long(), s["most"], torch.bfloat16
    slot, kept = torch.arange(len(s["expert"]), device="cuda"), s["expert"] < E
    place = torch.where(kept, s["expert"] * most + slot - off[s["expert"]], E * most)

    def table(rows):
        t = torch.zeros((E * most + 1, rows.shape[1]), device="cuda")
        t[place] = rows
        return t[:-1].view(E, most, rows.shape[1])

    def slots(t):
        return torch.where(kept[:, None], t.reshape(E * most, t.shape[2])[place.clamp_max(E * most - 1)], 0.0)

    wgu, wd = s["w_gateup"].float(), s["w_down"].float()
    out = {}
    if op in ("ffn", "step"):
        x = s["x_perm"].float() if op == "ffn" else s["x"].float()[s["token"]]
        a = torch.bmm(table(x), wgu.transpose(1, 2))
        g, u = a[:, :, :I], a[:, :, I:]
        h = g / (1 + torch.exp(-g)) * u
        out["y"] = slots(torch.bmm(h, wd.transpose(1, 2))).to(bf)
        a = slots(a)
        if c["act"] == "q8":
            a = torch.cat([_through_8_bits(a[:, :I]), _through_8_bits(a[:, I:])], 1)
        if op == "ffn":
            out["act"] = a.to(bf)
            return out
        x = _through_8_bits(s["x"])[s["token"]]
    else:
        x = s["x_perm"].float()
        if c["act"] == "q8":
            G = s["act_exp"].shape[1] // 2
            a = torch.cat([_values(s["act"][:, :I], s["act_exp"][:, :G]), _values(s["act"][:, I:], s["act_exp"][:, G:])], 1)
        else:
            a = s["act"].float()
    if c["act"] == "bf16" and op == "step":
        a = a.to(bf).float()
    dy = table(s["dy"].float())
    dh = slots(torch.bmm(dy, wd))
    g, u = a[:, :I], a[:, I:]
    sig = 1 / (1 + torch.exp(-g))
    da = table(torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1))
    out["dx"] = slots(torch.bmm(da, wgu)).to(bf)
    out["dw_gateup"] = torch.bmm(da.transpose(1, 2), table(x)).to(bf)
    out["dw_down"] = torch.bmm(dy.transpose(1, 2), table(g * sig * u)).to(bf)
    return out


def work(case):
    c = case
    T, H, E, I = c["T"], c["H"], c["E"], c["I"]
    op, wide = c["op"], 1 + 1 / GROUP
    if op == "checkpoint":
        a = 2 if c["rows"] == "bf16" else 4
        return {"bytes": 2 * T * H * (a + wide), "flops": 4 * T * H}
    R = T * c["k"] * (1 - c["drop"])
    if op == "restore":
        return {"bytes": T * H * wide + R * H * 2 + T * c["k"] * 4, "flops": R * H}
    used = E * (1 - (1 - min(1.0, c["k"] / E)) ** T) if c["zipf"] == 0 else min(E, R)  # experts that have rows
    act = R * 2 * I * (2 if c["act"] == "bf16" else wide)
    weights = 3 * H * I * 2
    forward = {"bytes": used * weights + 2 * R * H * 2 + act, "flops": 6 * R * H * I}
    backward = {"bytes": (used + E) * weights + 3 * R * H * 2 + act, "flops": 12 * R * H * I}
    if op == "ffn":
        return forward
    if op == "ffn_bwd":
        return backward
    kept = 2 * T * H * wide + T * H * 2 * 2
    return {"bytes": forward["bytes"] + backward["bytes"] + kept, "flops": forward["flops"] + backward["flops"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_power(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_8_bits(x):
    """The values of the 8-bit form, group by group of columns."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], GROUP):
        v = x[:, c:c + GROUP]
        m, p = torch.frexp(v.abs().max(1, keepdim=True).values / 127)
        scale = _exact_power(torch.where(m == 0.5, p - 1, p).clamp(-126, 121))
        out[:, c:c + GROUP] = torch.round(v / scale).clamp(-127, 127) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    op, E, I = case["op"], case["E"], case["I"]
    if op == "checkpoint":
        return {"out": _exact_8_bits(s["x"].to(f8))}
    if op == "restore":
        scale = _exact_power(s["exp"].to(torch.int64) - 127)
        v = torch.stack([s["q"][:, j].to(f8) * scale[:, j // GROUP] for j in range(case["H"])], 1)
        return {"x_perm": v[s["token"]] * (s["expert"] < E)[:, None]}
    off = s["offsets"].tolist()
    R = len(s["expert"])
    forward, backward = op in ("ffn", "step"), op in ("ffn_bwd", "step")
    new = lambda w: torch.zeros((R, w), device="cuda", dtype=f8)  # noqa: E731
    y, act, dx = new(case["H"] if forward else 0), new(2 * I), new(case["H"] if backward else 0)
    x = s["x"].to(f8)[s["token"]] if op == "step" else s["x_perm"].to(f8)
    if backward:
        # gradients are rounded to their type as they are stored: all experts' in 64 bits would be 20 GB
        f4 = torch.float32
        dwgu = torch.zeros(s["w_gateup"].shape, device="cuda", dtype=f4)
        dwd = torch.zeros(s["w_down"].shape, device="cuda", dtype=f4)
        xb = _exact_8_bits(s["x"].to(f8))[s["token"]] if op == "step" else x
    if op == "ffn_bwd":
        if case["act"] == "q8":
            G = s["act_exp"].shape[1] // 2
            scale = _exact_power(s["act_exp"].to(torch.int64) - 127)
            for j in range(2 * I):
                act[:, j] = s["act"][:, j].to(f8) * scale[:, j // GROUP if j < I else G + (j - I) // GROUP]
        else:
            act = s["act"].to(f8)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        wgu, wd = s["w_gateup"][e].to(f8), s["w_down"][e].to(f8)
        if forward:
            v = x[a:b] @ wgu.t()
            y[a:b] = (torch.sigmoid(v[:, :I]) * v[:, :I] * v[:, I:]) @ wd.t()
            if case["act"] == "q8":
                act[a:b] = torch.cat([_exact_8_bits(v[:, :I]), _exact_8_bits(v[:, I:])], 1)
            else:  # what the backward pass reads are bf16 values
                act[a:b] = v if op == "ffn" else v.to(torch.bfloat16).to(f8)
        if backward:
            g, u, d = act[a:b, :I], act[a:b, I:], s["dy"][a:b].to(f8)
            sg = torch.sigmoid(g)
            dh = d @ wd
            da = torch.cat([dh * u * (sg + g * sg * (1 - sg)), dh * sg * g], 1)
            dx[a:b] = da @ wgu
            dwgu[e] = (da.t() @ xb[a:b]).to(f4)
            dwd[e] = (d.t() @ (sg * g * u)).to(f4)
    out = {"y": y} if forward else {}
    if op == "ffn":
        # in 8 bits a value next to a border between two steps has no one value: it goes by the last bits of a sum
        out["act"] = None if case["act"] == "q8" else act
    if backward:
        out.update(dx=dx, dw_gateup=dwgu, dw_down=dwd)
    return out
