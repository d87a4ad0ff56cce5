"""Cases of the operators that feed the MoE expert FFN: the residual RMS norm with its 8-bit output
(``norm``), the router's product (``router``) and the gate that turns logits into expert ids and
weights (``gate``).

``run`` computes one of them in elementary torch operations, or, with ``own`` set, through the
library's entry points on the same state.
"""
import math

import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
TYPES = {"bf16": BF16, "f32": F32}
INF = float("inf")
EPS = 1e-6
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------- cases

def _norm(T, H, x="bf16", residual="bf16", weight="bf16", y=True, name=None):
    return _case(name, op="norm", T=T, H=H, x=x, residual=residual, weight=weight, y=y)


def _router(T, H, G, weight="bf16", name=None):
    return _case(name, op="router", T=T, H=H, G=G, weight=weight)


def _gate(T, G, k, score="softmax", bias=False, groups=1, kept=1, pair=False, renorm=True, scale=1.0, logits="f32",
          hole=0.0, name=None):
    return _case(name, op="gate", T=T, G=G, k=k, score=score, bias=bias, groups=groups, kept=kept, pair=pair,
                 renorm=renorm, scale=scale, logits=logits, hole=hole)


def _case(name, **kw):
    return dict(kw, name=name) if name else kw


def listed():
    return [
        # one token of a decoding batch: all latency
        _norm(1, 7168, name="norm one token"),
        # a decoding batch
        _norm(128, 7168, name="norm decode"),
        # a prompt of odd length, first layer (no residual yet), router fed elsewhere, FP32 weights
        _norm(2047, 4096, residual="none", weight="f32", y=False, name="norm ragged prompt"),
        # a large prefill batch
        _norm(16384, 7168, name="norm prefill"),
        # router of a decoding batch: the weights are most of what is read
        _router(128, 7168, 256, name="router decode"),
        # FP32 router weights, a tensor-parallel layer's 64 experts
        _router(2048, 4096, 64, weight="f32", name="router f32 weights"),
        # a large prefill batch
        _router(16384, 7168, 256, name="router prefill"),
        # all ranks' tokens at 384 experts
        _router(65536, 7168, 384, name="router all ranks"),
        # grouped sigmoid gate with a balance bias, decoding batch
        _gate(128, 256, 8, "sigmoid", True, 8, 4, True, True, 2.5, name="gate decode grouped"),
        # softmax gate on BF16 logits of a padded batch: rows and experts that are masked out
        _gate(2048, 64, 8, logits="bf16", hole=0.1, name="gate masked bf16"),
        # grouped sigmoid gate of a large prefill batch
        _gate(16384, 256, 8, "sigmoid", True, 8, 4, True, True, 2.5, name="gate prefill grouped"),
        # all ranks' tokens, ungrouped, balance bias
        _gate(65536, 384, 6, "sigmoid", True, name="gate all ranks"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "router", "gate"])
    if op == "norm":
        H = 32 * _log(rng, 2, 512)
        T = _log(rng, 1, min(65536, 16384 * 7168 // (2 * H)))
        return _norm(T, H, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32", "none"]),
                     rng.choice(["bf16", "f32"]), rng.random() < 0.7)
    if op == "router":
        H, G = 32 * _log(rng, 8, 256), _log(rng, 8, 512)
        w = rng.choice(["bf16", "bf16", "f32"])
        T = _log(rng, 1, min(65536, 65536 * 7168 * 384 // (H * G * (6 if w == "f32" else 1))))
        return _router(T, H, G, w)
    groups = rng.choice([1, 1, 4, 8])
    G = groups * _log(rng, max(4, 16 // groups), 512 // groups)
    kept = rng.randint(1, groups)
    k = rng.randint(1, min(16, G * kept // groups))
    return _gate(_log(rng, 1, min(65536, 65536 * 384 // G)), G, k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6,
                 groups, kept, rng.random() < 0.5, rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.choice(["f32", "bf16"]),
                 rng.choice([0.0, 0.1]))


# --------------------------------------------------------------------------------------- inputs

def _inputs(c, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=F32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    T = c["T"]
    if c["op"] == "norm":
        H = c["H"]
        x = normal(T, H)
        # a few channels and rows carry values far above the rest, as activations do
        x *= torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        x *= torch.where(torch.rand(T, 1, generator=g, device="cuda") < 0.1, 50.0, 1.0)
        d = {"x": x.to(TYPES[c["x"]]), "weight": (1 + 0.1 * normal(H)).to(TYPES[c["weight"]])}
        if c["residual"] != "none":
            d["residual"] = (4 * normal(T, H)).to(TYPES[c["residual"]])
        return d
    if c["op"] == "router":
        H, G = c["H"], c["G"]
        return {"x": normal(T, H).to(BF16), "weight": (normal(G, H) / H ** 0.5).to(TYPES[c["weight"]])}
    G = c["G"]
    logits = normal(T, G)
    if c["hole"]:  # padding rows, and experts that a row may not use
        drop = torch.rand(T, G, generator=g, device="cuda") < c["hole"]
        drop |= torch.rand(T, 1, generator=g, device="cuda") < c["hole"]
        logits.masked_fill_(drop, -INF)
    d = {"logits": logits.to(TYPES[c["logits"]])}
    if c["bias"]:  # a balance bias moves by fixed steps
        d["bias"] = torch.randint(-100, 101, (G,), generator=g, device="cuda").to(F32) * 1e-3
    return d


def prepare(case, seed):
    c = dict(case)
    d = _inputs(c, seed)
    state = {"case": c, **d}
    if own:
        state["call"], state["out"] = _bound(c, d)
    return state


def _bound(c, d):
    """The library's call with its output buffers, as a program that issues it again and again keeps it."""
    from moe_expert_ffn_plan_amd import binding as B

    T, dev = c["T"], "cuda"
    if c["op"] == "norm":
        H, r = c["H"], d.get("residual")
        s = B.make_norm(T, H, eps=EPS, x_dtype=TYPES[c["x"]], weight_dtype=TYPES[c["weight"]],
                        residual_dtype=BF16 if r is None else r.dtype)
        xq = torch.empty(T, H, dtype=torch.uint8, device=dev)
        xsf = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
        y = torch.empty(T, H, dtype=BF16, device=dev) if c["y"] else None
        rout = torch.empty_like(r) if r is not None else None
        call = B.norm_quant(s, d["x"], d["weight"], xq, xsf, y=y, residual=r, residual_out=rout, bind=True)
        out = {"q": xq.view(torch.float8_e4m3fn), "scale": xsf.view(torch.float8_e8m0fnu)}
        if y is not None:
            out["y"] = y
        if rout is not None:
            out["residual"] = rout
        return call, out
    if c["op"] == "router":
        s = B.make_router(T, c["H"], c["G"], weight_dtype=TYPES[c["weight"]])
        logits = torch.empty(T, c["G"], dtype=F32, device=dev)
        ws = torch.empty(B.router_workspace_bytes(s), dtype=torch.uint8, device=dev)
        return B.router_logits(s, d["x"], B.router_prepare(s, d["weight"]), logits, ws, bind=True), {"logits": logits}
    s = B.make_gate(T, c["G"], c["k"], score=c["score"], num_groups=c["groups"], topk_groups=c["kept"],
                    group_score="top2" if c["pair"] else "max", renormalize=c["renorm"], scale=c["scale"],
                    logits_dtype=TYPES[c["logits"]])
    ids = torch.empty(T, c["k"], dtype=torch.int64, device=dev)
    w = torch.empty(T, c["k"], dtype=F32, device=dev)
    return B.gate(s, d["logits"], ids, w, bias=d.get("bias"), bind=True), {"ids": ids, "weights": w}


def run(state):
    if own:
        state["call"]()
        return state["out"]
    return {"norm": _plain_norm, "router": _plain_router, "gate": _plain_gate}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------- plain forms

def _plain_norm(s):
    c = s["case"]
    h = s["x"].to(F32)
    out = {}
    if "residual" in s:
        h = h + s["residual"].to(F32)
        out["residual"] = h.to(s["residual"].dtype)
    v = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].to(F32)
    if c["y"]:
        out["y"] = v.to(BF16)
    b = v.view(c["T"], c["H"] // 32, 32)
    top = b.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)                 # 448 = 0.875 * 2^9
    e = torch.where(top > 0, e, -127).clamp(-127, 127)
    out["q"] = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).view(c["T"], c["H"])
    out["scale"] = torch.ldexp(torch.ones_like(top), e).to(torch.float8_e8m0fnu)
    return out


def _plain_router(s):
    return {"logits": s["x"].to(F32) @ s["weight"].to(F32).t()}


def _plain_gate(s):
    c = s["case"]
    T, G, k = c["T"], c["G"], c["k"]
    pair = c["pair"] and c["groups"] > 1
    # sums of scores and biases are compared with each other: in 32 bits their rounding would pick other experts
    logits = s["logits"].to(F64 if pair or "bias" in s else F32)
    off = logits == -INF
    if c["score"] == "softmax":
        top = logits.amax(-1, keepdim=True)
        e = torch.exp(logits - torch.where(top == -INF, 0.0, top))
        score = e / torch.where(top == -INF, 1.0, e.sum(-1, keepdim=True))
    else:
        score = 1 / (1 + torch.exp(-logits))
    # without a bias both scores rise with the logit, so the logits order them where the scores round alike
    order = score + s["bias"] if "bias" in s else logits
    if c["groups"] > 1:
        n = G // c["groups"]
        by = (score if pair and "bias" not in s else order).masked_fill(off, -INF).view(T, c["groups"], n)
        best = by.sort(dim=-1, descending=True).values
        mark = best[..., 0]
        if pair and n > 1:
            mark = mark + torch.where(best[..., 1] == -INF, 0.0, best[..., 1])
        keep = mark.sort(dim=-1, descending=True, stable=True).indices[:, : c["kept"]]
        held = torch.zeros_like(mark, dtype=torch.bool).scatter_(1, keep, True)
        off = off | ~held.repeat_interleave(n, 1)
    ids = order.masked_fill(off, -INF).sort(dim=-1, descending=True, stable=True).indices[:, :k]
    none = off.gather(1, ids)
    w = score.gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return {"ids": ids.masked_fill(none, -1), "weights": (w * c["scale"]).to(F32)}


# ------------------------------------------------------------------------------------------ work

def work(case):
    c = case
    T, size = c["T"], {"bf16": 2, "f32": 4, "none": 0}
    if c["op"] == "norm":
        H = c["H"]
        per = size[c["x"]] + 2 * size[c["residual"]] + (2 if c["y"] else 0) + 1 + 1 / 32
        return {"bytes": T * H * per + H * size[c["weight"]], "flops": 7 * T * H}
    if c["op"] == "router":
        H, G = c["H"], c["G"]
        return {"bytes": 2 * T * H + size[c["weight"]] * G * H + 4 * T * G, "flops": 2 * T * G * H}
    G, k = c["G"], c["k"]
    return {"bytes": T * G * size[c["logits"]] + (4 * G if c["bias"] else 0) + 12 * T * k, "flops": 5 * T * G}


# ----------------------------------------------------------------------------------------- exact

def exact(case, seed):
    d = _inputs(case, seed)
    return {"norm": _exact_norm, "router": _exact_router, "gate": _exact_gate}[case["op"]](case, d)


def _exact_norm(c, d):
    T, H = c["T"], c["H"]
    h = d["x"].double()
    out = {}
    if "residual" in d:
        h += d["residual"].double()
        out["residual"] = h
    v = h / (torch.linalg.vector_norm(h, dim=1) / H ** 0.5).square().add(EPS).sqrt()[:, None]
    v *= d["weight"].double()
    if c["y"]:
        out["y"] = v
    peak = v.abs().reshape(-1, 32).max(1).values
    # the smallest power of two that brings the peak to 448 or below, found by trying around log2
    p = torch.floor(torch.log2(peak.clamp_min(1e-300) / E4M3_MAX)) - 1
    for _ in range(3):
        p = torch.where(peak > E4M3_MAX * torch.exp2(p), p + 1, p)
    p = torch.where(peak == 0, torch.full_like(p, -127), p.clamp(-127, 127))
    scale = torch.exp2(p)
    # the value that an 8-bit code stands for, before its rounding to 8 bits
    out["q"] = (v.reshape(-1, 32) / scale[:, None]).reshape(T, H)
    out["scale"] = scale.reshape(T, H // 32)
    return out


def _exact_router(c, d):
    w = d["weight"].double().t().contiguous()
    return {"logits": torch.cat([x.double() @ w for x in d["x"].split(16384)])}


def _exact_gate(c, d):
    """Round after round: the largest value left, and the lowest place that has it."""
    T, G, k = c["T"], c["G"], c["k"]
    lg = d["logits"].double()
    alive = lg > -INF
    if c["score"] == "softmax":
        shift = torch.where(alive.any(1), lg.max(1).values, 0.0)
        p = (lg - shift[:, None]).exp() * alive
        p /= p.sum(1, keepdim=True).clamp_min(torch.finfo(F64).tiny)
    else:
        p = torch.where(lg >= 0, 1 / (1 + (-lg).exp()), lg.exp() / (1 + lg.exp())) * alive
    has_bias = "bias" in d
    key = p + d["bias"].double() if has_bias else lg

    def first_largest(v, ok):
        """(place, whether there is one) per row of the largest allowed value, the lowest place of equal ones."""
        v = torch.where(ok, v, -INF)
        hit = ok & (v == v.max(1, keepdim=True).values)
        place = torch.where(hit, torch.arange(v.shape[1], device=v.device), v.shape[1]).min(1).values
        return place.clamp_max(v.shape[1] - 1), ok.any(1)

    ok = alive
    if c["groups"] > 1:
        n = G // c["groups"]
        src = key if has_bias or not c["pair"] else p
        marks, live = [], []
        for q in range(c["groups"]):
            v, a = src[:, q * n:(q + 1) * n], alive[:, q * n:(q + 1) * n].clone()
            at, there = first_largest(v, a)
            mark = torch.where(there, v.gather(1, at[:, None])[:, 0], -INF)
            if c["pair"]:
                a[torch.arange(T, device=v.device), at] = False
                at, second = first_largest(v, a)
                mark = mark + torch.where(second, v.gather(1, at[:, None])[:, 0], 0.0)
            marks.append(mark)
            live.append(there)
        marks, live = torch.stack(marks, 1), torch.stack(live, 1)
        held = torch.zeros_like(live)
        for _ in range(c["kept"]):
            at, there = first_largest(marks, live)
            held[torch.arange(T, device=at.device)[there], at[there]] = True
            live = live & ~held
        ok = alive & held.repeat_interleave(n, 1)
    ids = torch.full((T, k), -1, dtype=torch.int64, device=lg.device)
    w = torch.zeros(T, k, dtype=F64, device=lg.device)
    ok = ok.clone()
    rows = torch.arange(T, device=lg.device)
    for j in range(k):
        at, there = first_largest(key, ok)
        ids[there, j] = at[there]
        w[there, j] = p[rows, at][there]
        ok[rows, at] = False
    if c["renorm"]:
        w = torch.where(w.sum(1, keepdim=True) > 0, w / w.sum(1, keepdim=True), 0.0)
    return {"ids": ids, "weights": w * c["scale"]}
