"""Cases of the operators around the 4-bit experts: microscaled quantisation (``quant``), the product of a dense
layer in 4 bits (``linear``), and the balance of the experts' load with its gradient (``balance`` and ``grad``).

``run`` computes one of them in elementary torch operations, or, with ``own`` set, through the library's entry
points on the same state.
"""
import math

import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
TYPES = {"bf16": BF16, "f32": F32}
INF = float("inf")
PEAK = {"e2m1": 6.0, "e4m3": 448.0}  # the largest value of a format


# ---------------------------------------------------------------------------------------- cases

def _quant(R, C, format="e2m1", x="bf16", wide=False, name=None):
    """wide: the columns are the first half of wider rows.  4-bit codes come with the values they stand for."""
    return _case(name, op="quant", R=R, C=C, format=format, x=x, wide=wide)


def _linear(T, K, N, format="e2m1", name=None):
    """e2m1: x is BF16 and quantised within the pass; e4m3: x is what a norm has quantised."""
    return _case(name, op="linear", T=T, K=K, N=N, format=format)


def _balance(T, E, k, score="softmax", seqs=1, logits="f32", hole=0.0, name=None):
    return _case(name, op="balance", T=T, E=E, k=k, score=score, seqs=seqs, logits=logits, hole=hole)


def _grad(T, E, k, score="softmax", seqs=1, logits="f32", hole=0.0, renorm=True, scale=1.0, weights=True, name=None):
    """weights: with the gradient of the gate's weights, else that of the loss alone."""
    return _case(name, op="grad", T=T, E=E, k=k, score=score, seqs=seqs, logits=logits, hole=hole, renorm=renorm,
                 scale=scale, weights=weights)


def _case(name, **kw):
    return dict(kw, name=name) if name else kw


def listed():
    return [
        # a decoding batch's activations in 4 bits, with the values they stand for (quantisation-aware training)
        _quant(128, 7168, name="quant decode"),
        # the gate half of a prefill batch's gate/up rows in 8 bits
        _quant(16384, 2048, "e4m3", wide=True, name="quant half rows"),
        # one token through a dense layer: the weights are all that is read
        _linear(1, 7168, 4096, "e4m3", name="linear one token"),
        # a decoding batch, activations in 4 bits
        _linear(128, 7168, 4096, name="linear decode"),
        # a prompt of odd length, a layer of odd width and a depth that no tile divides
        _linear(2047, 4064, 1537, "e4m3", name="linear ragged prompt"),
        # a large prefill batch
        _linear(16384, 7168, 4096, name="linear prefill"),
        # one small batch
        _balance(128, 256, 8, name="balance small"),
        # packed sequences of a prefill batch, some of them empty, with padding rows and masked experts
        _balance(16384, 256, 8, "sigmoid", 13, "bf16", 0.1, name="balance sequences"),
        # all ranks' tokens
        _balance(65536, 384, 6, name="balance all ranks"),
        # one small batch
        _grad(128, 64, 8, name="grad small"),
        # packed sequences, scaled sigmoid weights
        _grad(16384, 256, 8, "sigmoid", 13, "bf16", 0.1, True, 2.5, name="grad sequences"),
        # all ranks' tokens, weights that are not renormalised
        _grad(65536, 384, 6, renorm=False, name="grad all ranks"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "balance", "grad"])
    if op == "quant":
        C = 32 * _log(rng, 1, 512)
        return _quant(_log(rng, 1, max(1, min(65536, 16384 * 2048 // C))), C, rng.choice(["e2m1", "e4m3"]),
                      rng.choice(["bf16", "f32"]), rng.random() < 0.3)
    if op == "linear":
        K, N = 32 * _log(rng, 4, 256), _log(rng, 16, 8192)
        return _linear(_log(rng, 1, min(16384, 16384 * 7168 * 4096 // (2 * K * N))), K, N, rng.choice(["e2m1", "e4m3"]))
    E = _log(rng, 8, 512)
    T = _log(rng, 1, min(65536, 65536 * 384 // E))
    a = (T, E, rng.randint(1, min(16, E)), rng.choice(["softmax", "sigmoid"]), _log(rng, 1, 64), rng.choice(["f32", "bf16"]),
         rng.choice([0.0, 0.1]))
    return _balance(*a) if op == "balance" else _grad(*a, rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.random() < 0.7)


# --------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, T, C):
    """A few channels and rows carry values far above the rest."""
    x = torch.randn(T, C, generator=g, device="cuda")
    x *= torch.where(torch.rand(C, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    x *= torch.where(torch.rand(T, 1, generator=g, device="cuda") < 0.1, 50.0, 1.0)
    return x


def _inputs(c, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    g = _generator(seed)
    if c["op"] == "quant":
        x = _activations(g, c["R"], c["C"] * (2 if c["wide"] else 1)).to(TYPES[c["x"]])
        return {"x": x[:, :c["C"]]}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        x = _activations(g, T, K).to(BF16)
        d = {"x": x} if c["format"] == "e2m1" else dict(zip(("x", "x_sf"), _codes(x, "e4m3")))
        d["w"], d["w_sf"] = _codes(torch.randn(N, K, generator=g, device="cuda") / K ** 0.5, "e2m1")
        return d
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    # some experts are in favour, so that the load is uneven
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    if c["hole"]:  # padding rows, and experts that a row may not use
        drop = torch.rand(T, E, generator=g, device="cuda") < c["hole"]
        drop |= torch.rand(T, 1, generator=g, device="cuda") < c["hole"]
        logits.masked_fill_(drop, -INF)
    logits = logits.to(TYPES[c["logits"]])
    top = logits.to(F32).sort(dim=-1, descending=True, stable=True)
    d = {"logits": logits, "ids": top.indices[:, :k].masked_fill(top.values[:, :k] == -INF, -1).contiguous()}
    if S > 1:  # sequences end anywhere, and rows may be left behind the last
        cuts = torch.randint(0, T + 1, (S + 1,), generator=g, device="cuda").sort().values
        cuts[0] = 0
        d["offsets"] = cuts
    if c["op"] == "grad":
        seq = _sequences(d, T, S)
        d["counts"], d["rows"] = _counts(d["ids"], seq, E, S), _rows(logits, seq, S)
        d["d_loss"] = 1e-2 * (1 + torch.rand(S, generator=g, device="cuda"))
        d["d_z"] = 1e-3 * (1 + torch.rand(S, generator=g, device="cuda"))
        if c["weights"]:
            # a mean over the tokens: the size that the loss's own gradient has
            d["d_weights"] = torch.randn(T, k, generator=g, device="cuda") / T
        if c["score"] == "sigmoid":
            del d["d_z"]
    return d


def prepare(case, seed):
    c = dict(case)
    d = _inputs(c, seed)
    state = {"case": c, **d}
    if own:
        state["calls"], state["out"] = _bound(c, d)
    return state


def _bound(c, d):
    """The library's calls with their output buffers, as a program that issues them again and again keeps them."""
    from moe_expert_ffn_plan_amd import binding as B

    def empty(*shape, dtype=torch.uint8):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if c["op"] == "quant":
        R, C, four = c["R"], c["C"], c["format"] == "e2m1"
        s = B.make_mx_quant(R, C, format=c["format"], x_dtype=TYPES[c["x"]], x_stride=2 * C if c["wide"] else 0)
        q, sf = empty(R, C // 2 if four else C), empty(R, C // 32)
        dq = empty(R, C, dtype=BF16) if four else None
        out = {"scale": sf.view(torch.float8_e8m0fnu)}
        out.update({"values": dq} if four else {"q": q.view(torch.float8_e4m3fn)})
        return [B.mx_quant(s, d["x"], q, sf, x_dq=dq, bind=True)], out
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        s = B.make_mx_linear(T, K, N, x_format=c["format"])
        w = B.mx_linear_prepare(s, d["w"], d["w_sf"])
        ws = empty(B.mx_linear_workspace_bytes(s))
        y = empty(T, N, dtype=BF16)
        calls, q, sf = [], d["x"], d.get("x_sf")
        if c["format"] == "e2m1":
            q, sf = empty(T, K // 2), empty(T, K // 32)
            calls.append(B.mx_quant(B.make_mx_quant(T, K), d["x"], q, sf, bind=True))
        calls.append(B.mx_linear(s, q, sf, w, y, ws, bind=True))
        return calls, {"y": y}
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    s = B.make_balance(T, E, k, num_seqs=S, score=c["score"], logits_dtype=TYPES[c["logits"]],
                       renormalize=c.get("renorm", True), scale=c.get("scale", 1.0))
    if c["op"] == "balance":
        out = {"counts": empty(S, E, dtype=torch.int32), "rows": empty(S, dtype=torch.int32),
               "share": empty(S, E, dtype=F32), "loss": empty(S, dtype=F32)}
        if c["score"] == "softmax":
            out["z"] = empty(S, dtype=F32)
        return [B.balance(s, d["logits"], d["ids"], seq_offsets=d.get("offsets"), **out,
                          ws=empty(B.balance_workspace_bytes(s)), bind=True)], out
    out = {"logits": torch.zeros(T, E, dtype=TYPES[c["logits"]], device="cuda")}
    return [B.gate_grad(s, d["logits"], d["ids"], out["logits"], seq_offsets=d.get("offsets"), counts=d["counts"],
                        rows=d["rows"], d_loss=d["d_loss"], d_z=d.get("d_z"), d_topk_w=d.get("d_weights"), bind=True)], out


def run(state):
    if own:
        for call in state["calls"]:
            call()
        return state["out"]
    return {"quant": _plain_quant, "linear": _plain_linear, "balance": _plain_balance, "grad": _plain_grad}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------- plain forms

def _blocks(x, format):
    """x in blocks of 32 over their scales, and the scales' exponents: the smallest 2^e that brings a block's largest
    magnitude to the format's largest value or below."""
    b = x.to(F32).reshape(x.shape[0], -1, 32)
    top = b.abs().amax(-1)
    m, e = torch.frexp(top)
    full, at = (0.75, 3) if format == "e2m1" else (0.875, 9)  # 6 = 0.75 * 2^3, 448 = 0.875 * 2^9
    e = torch.where(m > full, e - at + 1, e - at)
    e = torch.where(top > 0, e, -127).clamp(-127, 127)
    v = torch.ldexp(b, -e[..., None])
    if format == "e2m1":
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
        v = torch.round(v / step) * step
    return v, e


def _codes(x, format):
    """x as stored: codes (two 4-bit ones to a byte, the even column low), and scales as their biased exponents."""
    v, e = _blocks(x, format)
    v = v.view(x.shape)
    if format == "e4m3":
        return v.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)
    a = v.abs()
    mag = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = mag | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _values(q, sf, format):
    """What stored codes and scales stand for, in 32 bits."""
    if format == "e4m3":
        v = q.view(torch.float8_e4m3fn).to(F32)
    else:
        code = torch.stack([q & 15, q >> 4], -1).flatten(1)
        mag = (code & 7).to(F32)
        v = torch.where(mag < 4, 0.5 * mag, torch.where(mag < 6, mag - 2, 2 * mag - 8))
        v = torch.where(code > 7, -v, v)
    return torch.ldexp(v.view(v.shape[0], -1, 32), sf.to(torch.int32)[..., None] - 127).view(v.shape)


def _plain_quant(s):
    c = s["case"]
    v, e = _blocks(s["x"], c["format"])
    out = {"scale": torch.ldexp(torch.ones_like(e, dtype=F32), e).to(torch.float8_e8m0fnu)}
    if c["format"] == "e2m1":
        out["values"] = torch.ldexp(v, e[..., None]).view(c["R"], c["C"]).to(BF16)
    else:
        out["q"] = v.view(c["R"], c["C"]).to(torch.float8_e4m3fn)
    return out


def _plain_linear(s):
    if s["case"]["format"] == "e2m1":
        v, e = _blocks(s["x"], "e2m1")
        x = torch.ldexp(v, e[..., None]).view(s["x"].shape)
    else:
        x = _values(s["x"], s["x_sf"], "e4m3")
    return {"y": (x @ _values(s["w"], s["w_sf"], "e2m1").t()).to(BF16)}


def _sequences(d, T, S):
    """The sequence of every row; S for rows that belong to none."""
    if "offsets" not in d:
        return torch.zeros(T, dtype=torch.int64, device="cuda")
    t = torch.arange(T, device="cuda")
    return torch.searchsorted(d["offsets"], t, right=True) - 1


def _counts(ids, seq, E, S):
    ok = (ids >= 0) & (seq < S)[:, None]
    at = torch.where(ok, seq[:, None] * E + ids, S * E)
    return torch.bincount(at.flatten(), minlength=S * E + 1)[:S * E].view(S, E).to(torch.int32)


def _rows(logits, seq, S):
    alive = (logits > -INF).any(-1)
    return torch.bincount(torch.where(alive, seq, S), minlength=S + 1)[:S].to(torch.int32)


def _shares(logits, score):
    """Every row's scores as shares of their sum, 0 throughout where all of them are masked, and the logarithm of the
    sum of exponentials."""
    top = logits.amax(-1, keepdim=True)
    alive = top > -INF
    top = torch.where(alive, top, 0.0)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    lse = torch.where(alive, top + torch.log(total), 0.0)
    if score == "sigmoid":
        e = 1 / (1 + torch.exp(-logits))
        total = e.sum(-1, keepdim=True)
    return e / torch.where(alive, total, 1.0), lse[:, 0]


def _plain_balance(s):
    c = s["case"]
    T, E, S = c["T"], c["E"], c["seqs"]
    logits = s["logits"].to(F32)
    seq = _sequences(s, T, S)
    counts, rows = _counts(s["ids"], seq, E, S), _rows(s["logits"], seq, S)
    p, lse = _shares(logits, c["score"])
    member = (seq[None] == torch.arange(S, device="cuda")[:, None]).to(F32)
    n = rows.clamp_min(1).to(F32)
    share = (member @ p) / n[:, None]
    total = counts.sum(-1).clamp_min(1)
    out = {"counts": counts, "rows": rows, "share": share, "loss": E * (counts * share).sum(-1) / total}
    if c["score"] == "softmax":
        out["z"] = (member @ (lse * lse)[:, None])[:, 0] / n
    return out


def _plain_grad(s):
    c = s["case"]
    T, E, S = c["T"], c["E"], c["seqs"]
    logits = s["logits"].to(F32)
    seq = _sequences(s, T, S)
    inside = (seq < S)[:, None]
    seq = seq.clamp_max(S - 1)
    p, lse = _shares(logits, c["score"])
    # a row's loss moves by its shares times these; what is the same for all experts falls out
    total = s["counts"].sum(-1, keepdim=True)
    pull = (s["counts"].to(torch.int64) * E - total) / total.clamp_min(1).to(F32)
    n = s["rows"].clamp_min(1).to(F32)
    pull = (pull * (s["d_loss"] / n)[:, None])[seq]
    away = 1 / (1 + torch.exp(logits))  # 1 - sigmoid
    grad = p * (pull - (p * pull).sum(-1, keepdim=True))
    if c["score"] == "sigmoid":
        grad = grad * away
    else:
        grad = grad + p * (2 * lse * (s["d_z"] / n)[seq])[:, None]
    if c["weights"]:
        ids = s["ids"].clamp_min(0)
        q = torch.where(s["ids"] >= 0, (p if c["score"] == "softmax" else 1 / (1 + torch.exp(-logits))).gather(1, ids), 0.0)
        dw = c["scale"] * s["d_weights"]
        if c["renorm"]:
            q = q / torch.where((s["ids"] >= 0).any(-1, keepdim=True), q.sum(-1, keepdim=True), 1.0)
            dw = dw - (q * dw).sum(-1, keepdim=True)
        g = q * dw
        if c["score"] == "sigmoid":
            g = g * away.gather(1, ids)
        elif not c["renorm"]:
            grad = grad - p * g.sum(-1, keepdim=True)
        grad = grad.scatter_add(1, ids, torch.where(s["ids"] >= 0, g, 0.0))
    return {"logits": torch.where(inside, grad, 0.0).to(s["logits"].dtype)}


# ------------------------------------------------------------------------------------------ work

def work(case):
    c, size = case, {"bf16": 2, "f32": 4}
    if c["op"] == "quant":
        out = 2.5 if c["format"] == "e2m1" else 1
        return {"bytes": c["R"] * c["C"] * (size[c["x"]] + out + 1 / 32), "flops": 3 * c["R"] * c["C"]}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": T * K * (2 if c["format"] == "e2m1" else 33 / 32) + N * K * 17 / 32 + 2 * T * N, "flops": 2 * T * K * N}
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    if c["op"] == "balance":
        return {"bytes": T * (E * size[c["logits"]] + 8 * k) + S * E * 8, "flops": 6 * T * E}
    return {"bytes": T * (2 * E * size[c["logits"]] + (12 if c["weights"] else 0) * k) + S * E * 4, "flops": 12 * T * E}


# ----------------------------------------------------------------------------------------- exact

def exact(case, seed):
    d = _inputs(case, seed)
    return {"quant": _exact_quant, "linear": _exact_linear, "balance": _exact_balance, "grad": _exact_grad}[case["op"]](case, d)


GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # E2M1's values by code


def _nearest(v, format):
    """The format's value next to each of v (none of them beyond its largest), the even code of two as near."""
    a = v.abs()
    if format == "e2m1":
        r = torch.zeros_like(a)
        for i in range(1, 8):
            half = (GRID[i - 1] + GRID[i]) / 2
            r = torch.where((a > half) | ((a == half) & (i % 2 == 0)), GRID[i], r)
    else:
        step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
        r = torch.round(a / step) * step
    return torch.copysign(r, v)


def _exact_blocks(x, format):
    """Rounded values over their scales, and the scales, found by trying the powers of two around."""
    b = x.double().reshape(-1, 32)
    peak = b.abs().max(1).values
    p = torch.floor(torch.log2(peak.clamp_min(1e-300) / PEAK[format])) - 1
    for _ in range(3):
        p = torch.where(peak > PEAK[format] * torch.exp2(p), p + 1, p)
    scale = torch.exp2(torch.where(peak == 0, torch.full_like(p, -127), p.clamp(-127, 127)))
    return _nearest(b / scale[:, None], format), scale


def _exact_quant(c, d):
    R, C = c["R"], c["C"]
    v, scale = _exact_blocks(d["x"], c["format"])
    out = {"scale": scale.view(R, C // 32)}
    if c["format"] == "e2m1":
        out["values"] = (v * scale[:, None]).view(R, C)
    else:
        out["q"] = v.view(R, C)
    return out


def _decoded(q, sf, format):
    if format == "e4m3":
        v = q.view(torch.float8_e4m3fn).double()
    else:
        grid = torch.tensor(GRID + [-g for g in GRID], dtype=F64, device=q.device)
        v = torch.empty(q.shape[0], 2 * q.shape[1], dtype=F64, device=q.device)
        v[:, 0::2], v[:, 1::2] = grid[(q % 16).long()], grid[(q // 16).long()]
    return v * torch.exp2(sf.double() - 127).repeat_interleave(32, 1)


def _exact_linear(c, d):
    w = _decoded(d["w"], d["w_sf"], "e2m1").t().contiguous()
    if c["format"] == "e2m1":
        v, scale = _exact_blocks(d["x"], "e2m1")
        x = (v * scale[:, None]).view(d["x"].shape)
    else:
        x = _decoded(d["x"], d["x_sf"], "e4m3")
    return {"y": torch.cat([r @ w for r in x.split(4096)])}


def _spans(c, d):
    at = [0, c["T"]] if "offsets" not in d else d["offsets"].tolist()
    return list(zip(at, at[1:]))


def _exact_shares(lg, score):
    alive = (lg > -INF).any(1)
    lse = torch.where(alive, torch.logsumexp(lg, 1), 0.0)
    if score == "softmax":
        return torch.where(alive[:, None], torch.softmax(lg, 1), 0.0), lse, alive
    sg = torch.sigmoid(lg)
    return torch.where(alive[:, None], sg / sg.sum(1, keepdim=True).clamp_min(1e-300), 0.0), lse, alive


def _exact_balance(c, d):
    S, E = c["seqs"], c["E"]
    p, lse, alive = _exact_shares(d["logits"].double(), c["score"])
    out = {"counts": torch.zeros(S, E, dtype=torch.int32), "rows": torch.zeros(S, dtype=torch.int32),
           "share": torch.zeros(S, E, dtype=F64), "loss": torch.zeros(S, dtype=F64), "z": torch.zeros(S, dtype=F64)}
    for i, (a, b) in enumerate(_spans(c, d)):
        n = int(alive[a:b].sum())
        ids = d["ids"][a:b].flatten()
        counts = torch.stack([(ids == e).sum() for e in range(E)]).cpu()
        out["counts"][i], out["rows"][i] = counts.to(torch.int32), n
        if n:
            out["share"][i] = p[a:b].sum(0).cpu() / n
            out["z"][i] = lse[a:b].square().sum().cpu() / n
        if counts.sum():
            out["loss"][i] = E * (counts.double() / counts.sum()) @ out["share"][i]
    if c["score"] == "sigmoid":
        del out["z"]
    return out


def _exact_grad(c, d):
    """The derivative by torch of the loss and of the weights, written down in 64 bits."""
    lg = d["logits"].double()
    dead = ~(lg > -INF)
    x = lg.masked_fill(dead, 0.0).requires_grad_()
    masked = x.masked_fill(dead, -1e6)  # exp gives 0, and so does its derivative
    alive = (~dead).any(1)
    if c["score"] == "softmax":
        p = torch.softmax(masked, 1)
    else:
        sg = torch.sigmoid(masked)
        p = sg / sg.sum(1, keepdim=True).clamp_min(1e-300)
    p = p * alive[:, None]
    total = 0.0
    for i, (a, b) in enumerate(_spans(c, d)):
        n = int(alive[a:b].sum())
        f = d["counts"][i].double()
        if n and f.sum():
            total = total + d["d_loss"][i].double() * c["E"] * ((f / f.sum()) * p[a:b].sum(0)).sum() / n
        if n and "d_z" in d:
            total = total + d["d_z"][i].double() * (torch.logsumexp(masked[a:b], 1).square() * alive[a:b]).sum() / n
    if c["weights"]:
        picked = d["ids"] >= 0
        inside = torch.zeros(c["T"], 1, dtype=F64, device="cuda")
        spans = _spans(c, d)
        inside[spans[0][0]:spans[-1][1]] = 1
        w = (p if c["score"] == "softmax" else sg).gather(1, d["ids"].clamp_min(0)) * picked
        if c["renorm"]:
            w = w / torch.where(picked.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
        total = total + c["scale"] * (w * d["d_weights"].double() * inside).sum()
    if not torch.is_tensor(total):  # no sequence has a row
        return {"logits": torch.zeros_like(lg)}
    return {"logits": torch.autograd.grad(total, x)[0].masked_fill(dead, 0.0)}
