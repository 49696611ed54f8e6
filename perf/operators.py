"""Cases for the operators around an expert layer: routing by scores, the experts' matrix products,
and the gradients that a training step takes through them.

Each case names its operator in "op":

  route            ids and gates of moe_route_scored
  route_backward   gradient of the logits (moe_route_scored_backward)
  matmul           rows of every expert times its weights, bias, activation, residual (moe_expert_matmul)
  matmul_backward  gradients of rows, weights and bias (moe_expert_matmul_backward)
  combine_backward gradients of the expert outputs and of the gates (moe_combine_backward)

`own` False computes the plain form with elementary torch operations; `own` True makes the calls a
program makes of the framework.  Rows that hold no token are never written: both forms return buffers
whose other rows are zero.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "swiglu")


def listed():
    return [
        # a decode step's router: 128 tokens, sigmoid scores, balance bias, 4 of 8 groups
        {"name": "route decode", "op": "route", "T": 128, "E": 256, "k": 8, "func": "sigmoid", "groups": 8,
         "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "bias": True},
        # a long prompt's router over 512 fine-grained experts
        {"name": "route fine-grained", "op": "route", "T": 65536, "E": 512, "k": 10, "func": "sigmoid",
         "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5, "bias": True},
        # a training step's router gradient, sigmoid scores renormalised over the chosen experts
        {"name": "route gradient", "op": "route_backward", "T": 32768, "E": 256, "k": 8, "func": "sigmoid",
         "renorm": True, "scale": 2.5},
        # softmax over all experts without renormalisation: every logit has a gradient; an odd batch
        {"name": "route gradient softmax", "op": "route_backward", "T": 4099, "E": 128, "k": 8,
         "func": "softmax", "renorm": False, "scale": 1.0},
        # serving one token: 8 of 256 experts' gate and up weights are read once
        {"name": "experts one token", "op": "matmul", "T": 1, "E": 256, "k": 8, "K": 7168, "F": 1024,
         "act": "swiglu", "bias": False, "residual": False, "save": False, "align": 1, "cap": 0, "skew": 0.0},
        # a decode batch's second product: nearly every expert has a few rows
        {"name": "experts decode", "op": "matmul", "T": 128, "E": 256, "k": 8, "K": 1024, "F": 7168,
         "act": "none", "bias": False, "residual": False, "save": False, "align": 1, "cap": 0, "skew": 0.0},
        # a prompt's (or a training step's) first product: 256 rows an expert, pre-activations kept
        {"name": "experts prefill", "op": "matmul", "T": 4096, "E": 128, "k": 8, "K": 4096, "F": 1024,
         "act": "swiglu", "bias": False, "residual": False, "save": True, "align": 1, "cap": 0, "skew": 0.3},
        # the always-on shared expert as one dense product over an odd batch, with bias, gelu and residual
        {"name": "shared expert", "op": "matmul", "T": 16387, "E": 1, "k": 1, "K": 2048, "F": 2048,
         "act": "gelu", "bias": True, "residual": True, "save": False, "align": 1, "cap": 0, "skew": 0.0},
        # a training step's gradients of the first product
        {"name": "experts gradient", "op": "matmul_backward", "T": 4096, "E": 128, "k": 8, "K": 4096, "F": 1024,
         "act": "swiglu", "bias": True, "align": 1, "cap": 0, "skew": 0.3},
        # gradients at small odd sizes, segments padded to 16 rows
        {"name": "experts gradient small", "op": "matmul_backward", "T": 299, "E": 16, "k": 2, "K": 520,
         "F": 264, "act": "gelu", "bias": True, "align": 16, "cap": 0, "skew": 0.3},
        # a training step's gradient through the combine
        {"name": "combine gradient", "op": "combine_backward", "T": 4096, "E": 128, "k": 8, "H": 4096,
         "align": 1, "cap": 0, "skew": 0.3},
        # a small batch with expert capacity: some slots are dropped
        {"name": "combine gradient capacity", "op": "combine_backward", "T": 130, "E": 64, "k": 8, "H": 7168,
         "align": 1, "cap": 16, "skew": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "matmul", "matmul", "matmul_backward", "combine_backward"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 4, 8, 16])
        E = groups * rng.randint(max(2, 16 // groups), 512 // groups)
        top = groups if groups == 1 else rng.randint(max(1, groups // 4), groups)
        k = rng.randint(1, min(16, top * (E // groups)))
        c = {"op": op, "T": _log_int(rng, 1, 32768), "E": E, "k": k, "func": rng.choice(["softmax", "sigmoid"]),
             "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5])}
        if op == "route":
            c.update(groups=groups, top_groups=top, group_top=rng.choice([1, 2]), bias=rng.random() < 0.7)
        return c
    E = rng.choice([1, 4, 8, 16, 32, 64])
    k = 1 if E == 1 else rng.randint(1, min(8, E))
    align = rng.choice([1, 1, 1, 16, 128])
    cap = 0
    T = _log_int(rng, 1, 4096)
    if align == 1 and rng.random() < 0.25:
        cap = max(1, int(T * k / E * rng.uniform(0.7, 1.5)))
    c = {"op": op, "T": T, "E": E, "k": k, "align": align, "cap": cap, "skew": rng.choice([0.0, 0.3, 0.6])}
    if op == "combine_backward":
        c["H"] = 8 * _log_int(rng, 8, 896)
        return c
    c.update(K=8 * _log_int(rng, 8, 512), F=8 * _log_int(rng, 8, 256), act=rng.choice(ACTS),
             bias=rng.random() < 0.5)
    if op == "matmul":
        c.update(residual=rng.random() < 0.4, save=rng.random() < 0.3)
    return c


# ---- sizes -----------------------------------------------------------------------------------------

def _rows(c):
    return c["E"] * c["cap"] if c["cap"] else c["T"] * c["k"] + c["E"] * (c["align"] - 1)


def _kept(c):
    """Rows that hold a token, about: all assignments, fewer with a capacity below the mean load."""
    return min(c["T"] * c["k"], c["E"] * c["cap"]) if c["cap"] else c["T"] * c["k"]


def _active(c):
    """Experts that get at least one token, expected for a uniform router."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def _wide(c):
    return 2 * c["F"] if c["act"] == "swiglu" else c["F"]


def work(case):
    c = case
    op, T = c["op"], c["T"]
    if op == "route":
        return {"bytes": T * c["E"] * 4 + T * c["k"] * 8 + (c["E"] * 4 if c["bias"] else 0), "flops": T * c["E"] * 6}
    if op == "route_backward":
        dense = c["func"] == "softmax" and not c["renorm"]
        read = T * (c["E"] if dense else c["k"]) * 4
        return {"bytes": read + T * c["k"] * 8 + T * c["E"] * 4, "flops": T * (c["E"] if dense else c["k"]) * 8}
    n = _kept(c)
    if op == "combine_backward":
        return {"bytes": T * c["H"] * 2 + n * c["H"] * 4 + T * c["k"] * 12, "flops": n * c["H"] * 3}
    K, F, W = c["K"], c["F"], _wide(c)
    weights = _active(c) * W * K * 2
    if op == "matmul":
        return {"bytes": weights + n * K * 2 + n * F * 2 + (n * W * 2 if c["save"] else 0)
                + (n * F * 2 if c["residual"] else 0) + (c["E"] * W * 4 if c["bias"] else 0),
                "flops": 2 * n * W * K}
    pre = n * W * 2 if c["act"] != "none" else 0
    return {"bytes": weights + c["E"] * W * K * 2 + n * F * 2 + pre + 2 * n * K * 2
            + (c["E"] * W * 4 if c["bias"] else 0), "flops": 4 * n * W * K}


# ---- inputs ----------------------------------------------------------------------------------------

def _layout(c, g, dev):
    """ids of a router with mildly uneven popularity, and the expert-major layout of their rows."""
    T, E, k = c["T"], c["E"], c["k"]
    pop = torch.randn(E, generator=g, device=dev) * c["skew"]
    ids = torch.topk(torch.randn(T, E, generator=g, device=dev) + pop, k, dim=1).indices
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    if c["cap"]:
        kept, seg = counts.clamp(max=c["cap"]), torch.full_like(counts, c["cap"])
    else:
        kept, seg = counts, (counts + c["align"] - 1) // c["align"] * c["align"]
    off = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    off[1:] = torch.cumsum(seg, 0)
    order = torch.argsort(flat, stable=True)
    first = torch.cumsum(counts, 0) - counts
    place = torch.empty_like(flat)
    place[order] = torch.arange(T * k, device=dev) - first[flat[order]]
    dst = torch.where(place < kept[flat], off[flat] + place, torch.full_like(flat, -1)).reshape(T, k)
    return counts, kept, off, dst


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op, T, E, k = c["op"], c["T"], c["E"], c["k"]

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    s = {"case": c}
    if op in ("route", "route_backward"):
        s["logits"] = normal(T, E, scale=1.5, dtype=torch.float32)
        if op == "route":
            s["bias"] = normal(E, scale=0.05, dtype=torch.float32) if c["bias"] else None
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
            s["gates"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        else:
            s["ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
            s["grad_gates"] = normal(T, k, dtype=torch.float32)
            s["grad_logits"] = torch.empty(T, E, dtype=torch.float32, device=dev)
        return s
    N = _rows(c)
    counts, kept, off, dst = _layout(c, g, dev)
    s["counts"], s["off"] = counts.to(torch.int32), off.to(torch.int32)
    if op == "combine_backward":
        s["dst"] = dst.to(torch.int32)
        s["y"], s["grad_out"] = normal(N, c["H"]), normal(T, c["H"])
        s["gates"] = torch.softmax(normal(T, k, dtype=torch.float32), 1)
        s["grad_y"] = torch.zeros(N, c["H"], dtype=torch.bfloat16, device=dev)
        s["grad_gates"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        return s
    K, F, W = c["K"], c["F"], _wide(c)
    # the plain form's plan: the experts with rows, and their row numbers padded to the longest (N: none)
    active = torch.nonzero(kept).reshape(-1)
    most = int(kept.max())
    at = torch.arange(most, device=dev)
    s["active"] = active
    s["slots"] = torch.where(at < kept[active][:, None], off[active][:, None] + at, torch.full_like(at, N))
    s["x"] = normal(N, K)
    s["w"] = normal(E, W, K, scale=1.0 / math.sqrt(K))
    bias = normal(E, W, scale=0.2, dtype=torch.float32) if c["bias"] else None
    if op == "matmul":
        s["bias"] = bias
        s["residual"] = normal(N, F) if c["residual"] else None
        s["out"] = torch.zeros(N, F, dtype=torch.bfloat16, device=dev)
        s["pre"] = torch.zeros(N, W, dtype=torch.bfloat16, device=dev) if c["save"] else None
        return s
    s["pre"] = normal(N, W) if c["act"] != "none" else None
    s["grad_out"] = normal(N, F)
    s["grad_x"] = torch.zeros(N, K, dtype=torch.bfloat16, device=dev)
    s["grad_w"] = torch.empty(E, W, K, dtype=torch.bfloat16, device=dev)
    s["grad_bias"] = torch.empty(E, W, dtype=torch.float32, device=dev) if c["bias"] else None
    return s


# ---- the plain forms -------------------------------------------------------------------------------

def _scores(c, logits):
    if c["func"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    # 64 bits: near-equal keys decide which expert is taken
    score = _scores(c, s["logits"].double())
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["top_groups"] < G:
        best = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True).values
        group = best[:, :, : c["group_top"]].sum(2)
        taken = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        allowed = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, taken, True)
        key = torch.where(allowed[:, :, None].expand(T, G, E // G).reshape(T, E), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    gates = torch.gather(score, 1, ids)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "gates": (gates * c["scale"]).float()}


def _route_backward(s):
    c = s["case"]
    ids, up = s["ids"].long(), s["grad_gates"] * c["scale"]
    logits = s["logits"]
    if c["func"] == "softmax" and not c["renorm"]:
        p = _scores(c, logits)
        d = torch.zeros_like(p).scatter_(1, ids, up)
        return {"grad_logits": p * (d - (d * p).sum(1, keepdim=True))}
    chosen = torch.gather(logits, 1, ids)
    if c["func"] == "softmax":
        q = _scores(c, chosen)
        d = q * (up - (up * q).sum(1, keepdim=True))
    else:
        v = _scores(c, chosen)
        d = up
        if c["renorm"]:
            total = v.sum(1, keepdim=True)
            d = (up - (up * v).sum(1, keepdim=True) / total) / total
        d = d * v * (1.0 - v)
    return {"grad_logits": torch.zeros_like(logits).scatter_(1, ids, d)}


def _by_expert(rows, slots):
    """The rows of each active expert in 32 bits, padded with zero rows: [A, longest, columns]."""
    padded = torch.cat([rows, rows.new_zeros(1, rows.shape[1])])
    return padded[slots].float()


def _to_rows(values, slots, n):
    out = torch.zeros(n + 1, values.shape[2], dtype=torch.bfloat16, device=values.device)
    out[slots.reshape(-1)] = values.reshape(-1, values.shape[2]).to(torch.bfloat16)
    return out[:n]


def _act(z, act, F):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "swiglu":
        gate, up = z[..., :F], z[..., F:]
        return gate / (1.0 + torch.exp(-gate)) * up
    return z


def _act_backward(z, d, act, F):
    if act == "relu":
        return d * (z > 0)
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return d * (cdf + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi))
    if act == "silu":
        v = 1.0 / (1.0 + torch.exp(-z))
        return d * v * (1.0 + z * (1.0 - v))
    if act == "swiglu":
        gate, up = z[..., :F], z[..., F:]
        v = 1.0 / (1.0 + torch.exp(-gate))
        return torch.cat([d * up * v * (1.0 + gate * (1.0 - v)), d * gate * v], -1)
    return d


def _matmul(s):
    c = s["case"]
    n, act, slots, active = s["x"].shape[0], c["act"], s["slots"], s["active"]
    z = torch.bmm(_by_expert(s["x"], slots), s["w"][active].float().transpose(1, 2))
    if s["bias"] is not None:
        z += s["bias"][active][:, None, :]
    y = _act(z, act, c["F"])
    if s["residual"] is not None:
        y = y + _by_expert(s["residual"], slots)
    got = {"out": _to_rows(y, slots, n)}
    if s["pre"] is not None:
        got["pre"] = _to_rows(z, slots, n)
    return got


def _matmul_backward(s):
    c = s["case"]
    n, slots, active = s["x"].shape[0], s["slots"], s["active"]
    d = _by_expert(s["grad_out"], slots)
    if s["pre"] is not None:
        d = _act_backward(_by_expert(s["pre"], slots), d, c["act"], c["F"])
    grad_x = torch.bmm(d, s["w"][active].float())
    grad_w = torch.zeros_like(s["w"])
    grad_w[active] = torch.bmm(d.transpose(1, 2), _by_expert(s["x"], slots)).to(torch.bfloat16)
    got = {"grad_x": _to_rows(grad_x, slots, n), "grad_w": grad_w}
    if s["grad_bias"] is not None:
        got["grad_bias"] = torch.zeros_like(s["grad_bias"])
        got["grad_bias"][active] = d.sum(1)
    return got


def _combine_backward(s):
    n = s["y"].shape[0]
    dst = s["dst"].long()
    held = dst >= 0
    out = s["grad_out"].float()
    rows = s["y"][dst.clamp(min=0)].float()
    grad_gates = (rows * out[:, None, :]).sum(2) * held
    grad_y = torch.zeros(n + 1, out.shape[1], dtype=torch.bfloat16, device=out.device)
    values = (s["gates"][:, :, None] * out[:, None, :]).to(torch.bfloat16)
    grad_y[torch.where(held, dst, torch.full_like(dst, n)).reshape(-1)] = values.reshape(-1, out.shape[1])
    return {"grad_y": grad_y[:n], "grad_gates": grad_gates}


PLAIN = {"route": _route, "route_backward": _route_backward, "matmul": _matmul,
         "matmul_backward": _matmul_backward, "combine_backward": _combine_backward}


# ---- the framework's calls -------------------------------------------------------------------------

_workspaces = {}


def _own(s):
    import combine_moe_route_07_b200 as m

    c = s["case"]
    op = c["op"]
    if "call" not in s:
        hidden = c.get("H") or c.get("K") or 8
        shape = m.MoeShape(tokens=c["T"], hidden=hidden, experts=c["E"], k=c["k"], ranks=1,
                           capacity=c.get("cap", 0), align=c.get("align", 1), renorm=c.get("renorm", True))
        rule = None
        if op in ("route", "route_backward"):
            rule = m.ScoreRule(func=c["func"], groups=c.get("groups", 1), top_groups=c.get("top_groups", 1),
                               group_top=c.get("group_top", 1), scale=c["scale"])
        # a program keeps one workspace for each problem size
        if shape not in _workspaces:
            _workspaces[shape] = m.Workspace(shape)
        s["call"] = (shape, _workspaces[shape], rule)
    shape, ws, rule = s["call"]
    if op == "route":
        ids, gates = m.moe_route_scored(shape, s["logits"], rule, s["bias"], ws=ws, ids=s["ids"], gates=s["gates"])
        return {"ids": ids, "gates": gates}
    if op == "route_backward":
        return {"grad_logits": m.moe_route_scored_backward(shape, s["logits"], rule, s["ids"], s["grad_gates"], ws=ws,
                                                           grad_logits=s["grad_logits"])}
    if op == "matmul":
        y = m.moe_expert_matmul(shape, s["x"], s["w"], s["counts"], s["off"], ws=ws, bias=s["bias"], act=c["act"],
                                residual=s["residual"], out=s["out"], pre=s["pre"])
        return {"out": y} if s["pre"] is None else {"out": y, "pre": s["pre"]}
    if op == "matmul_backward":
        g = m.moe_expert_matmul_backward(shape, s["grad_out"], s["x"], s["w"], s["counts"], s["off"], ws=ws,
                                         act=c["act"], pre=s["pre"], grad_x=s["grad_x"], grad_w=s["grad_w"],
                                         grad_bias=s["grad_bias"])
        got = {"grad_x": g.grad_x, "grad_w": g.grad_w}
        if s["grad_bias"] is not None:
            got["grad_bias"] = g.grad_bias
        return got
    grad_y, grad_gates = m.moe_combine_backward(shape, s["grad_out"], s["y"], s["dst"], s["gates"], ws=ws,
                                                grad_y=s["grad_y"], grad_gates=s["grad_gates"])
    return {"grad_y": grad_y, "grad_gates": grad_gates}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- the definitions in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    op, T, E = c["op"], c["T"], c["E"]
    if op in ("route", "route_backward"):
        z = s["logits"].double()
        score = torch.sigmoid(z) if c["func"] == "sigmoid" else torch.softmax(z, 1)
    if op == "route":
        key = score.clone()
        if s["bias"] is not None:
            key += s["bias"].double()
        size = E // c["groups"]
        if c["top_groups"] < c["groups"]:
            sums = []
            for q in range(c["groups"]):
                part = key[:, q * size:(q + 1) * size]
                sums.append(torch.topk(part, c["group_top"], dim=1).values.sum(1))
            order = torch.sort(-torch.stack(sums, 1), dim=1, stable=True).indices
            for r in range(c["top_groups"], c["groups"]):
                cols = order[:, r:r + 1] * size + torch.arange(size, device=z.device)
                key.scatter_(1, cols, -math.inf)
        ids = torch.sort(-key, dim=1, stable=True).indices[:, : c["k"]]
        g = score.gather(1, ids)
        g = g / g.sum(1, keepdim=True) if c["renorm"] else g
        return {"ids": None, "gates": g * c["scale"]}
    if op == "route_backward":
        ids = s["ids"].long()
        one = torch.zeros(T, c["k"], E, dtype=torch.float64, device=z.device) if T * c["k"] * E < 1 << 28 else None
        chosen = score.gather(1, ids)
        up = s["grad_gates"].double() * c["scale"]
        if c["renorm"]:  # gate = score / sum of the chosen scores
            total = chosen.sum(1, keepdim=True)
            up = up / total - (up * chosen).sum(1, keepdim=True) / total ** 2
        if c["func"] == "sigmoid":
            return {"grad_logits": torch.zeros_like(z).scatter_add_(1, ids, up * chosen * (1 - chosen))}
        if one is None:  # d score_j / d logit_e = score_j ([j = e] - score_e)
            got = torch.zeros_like(z).scatter_add_(1, ids, up * chosen)
            return {"grad_logits": got - score * (up * chosen).sum(1, keepdim=True)}
        one.scatter_(2, ids[:, :, None], 1.0)
        one -= score[:, None, :]
        one *= (up * chosen)[:, :, None]
        return {"grad_logits": one.sum(1)}
    off, kept = s["off"].tolist(), s["counts"].tolist()
    if c["cap"]:
        kept = [min(v, c["cap"]) for v in kept]
    if op == "combine_backward":
        dst = s["dst"].long()
        grad_y = torch.zeros(s["y"].shape, dtype=torch.float64, device=dst.device)
        grad_gates = torch.zeros(T, c["k"], dtype=torch.float64, device=dst.device)
        for j in range(c["k"]):
            t = torch.nonzero(dst[:, j] >= 0).reshape(-1)
            p, o = dst[t, j], s["grad_out"][t].double()
            grad_y[p] = s["gates"][t, j].double()[:, None] * o
            grad_gates[t, j] = torch.einsum("th,th->t", s["y"][p].double(), o)
        return {"grad_y": grad_y, "grad_gates": grad_gates}
    F, W, act = c["F"], _wide(c), c["act"]
    n, K = s["x"].shape
    if op == "matmul":
        out = torch.zeros(n, F, dtype=torch.float64, device=s["x"].device)
        pre = torch.zeros(n, W, dtype=torch.float64, device=s["x"].device) if c["save"] else None
        for e in range(E):
            r = slice(off[e], off[e] + kept[e])
            if kept[e]:
                z = s["x"][r].double() @ s["w"][e].double().T
                if s["bias"] is not None:
                    z = z + s["bias"][e].double()
                if pre is not None:
                    pre[r] = z
                if act == "relu":
                    z = z.clamp(min=0)
                elif act == "gelu":
                    z = z * torch.special.ndtr(z)
                elif act == "silu":
                    z = z * torch.sigmoid(z)
                elif act == "swiglu":
                    z = z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:]
                out[r] = z if s["residual"] is None else z + s["residual"][r].double()
        return {"out": out} if pre is None else {"out": out, "pre": pre}
    grad_x = torch.zeros(n, K, dtype=torch.float64, device=s["x"].device)
    grad_w = torch.zeros(E, W, K, dtype=torch.float64, device=s["x"].device)
    grad_b = torch.zeros(E, W, dtype=torch.float64, device=s["x"].device)
    for e in range(E):
        r = slice(off[e], off[e] + kept[e])
        if kept[e]:
            d = s["grad_out"][r].double()
            if act != "none":
                z = s["pre"][r].double()
                if act == "relu":
                    d = torch.where(z > 0, d, 0.0)
                elif act == "gelu":
                    d = d * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
                else:
                    a = z[:, :F]
                    v = torch.sigmoid(a)
                    slope = v + a * v * torch.sigmoid(-a)
                    d = d * slope if act == "silu" else torch.cat([d * z[:, F:] * slope, d * a * v], 1)
            grad_x[r] = d @ s["w"][e].double()
            grad_w[e] = d.T @ s["x"][r].double()
            grad_b[e] = d.sum(0)
    got = {"grad_x": grad_x, "grad_w": grad_w}
    if s["grad_bias"] is not None:
        got["grad_bias"] = grad_b
    return got
