"""GPU parity of moe_balance and moe_gate_grad with the float64 oracle.

A row's shares: the argument of the exponential is rounded once (2^-24 of up to 16 for these normal logits and their
distances), the exponential, the sum and the division add 2^-24 each a few times: SHARE = 2^-19 relative.  Sums over
rows of values of one sign add 2^-24 per level: a lane's run of at most 64 rows here, 6 levels of lanes and waves,
and the tiles: SUM = 2^-17.  Gradients are differences: the bound is relative to the magnitudes that are
subtracted, p * (|g| + mean of |g|) and the weights' counterpart.
"""
import itertools

import numpy as np
import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B
from oracle.balance import balance_ref, gate_grad_ref, row_scores, row_shares, spans
from oracle.front import gate_ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
SHARE, SUM = 2.0 ** -19, 2.0 ** -17


def inputs(T, E, k, seed, dtype=F32, hole=0.0, S=1, scale=1.0):
    """(logits, ids, offsets or None) on the host: uneven load, masked experts and padding rows, ids of -1."""
    g = np.random.default_rng(seed)
    l = torch.from_numpy((g.normal(size=(T, E)) + 0.5 * g.normal(size=E)) * scale).to(dtype)
    if hole:
        l[torch.from_numpy((g.random((T, E)) < hole) | (g.random((T, 1)) < hole))] = -INF
    v, ids = l.float().sort(dim=1, descending=True, stable=True)
    ids = torch.where(v[:, :k] == -INF, -1, ids[:, :k])
    off = None
    if S > 1:
        off = torch.from_numpy(np.sort(g.integers(0, T + 1, S + 1)))
    return l, ids.contiguous(), off


def forward(l, ids, off, gpu, score="softmax", S=1, stride=0, only=None, shape=None):
    T, E = l.shape
    s = shape or B.make_balance(T, E, ids.shape[1], num_seqs=S, score=score, logits_dtype=l.dtype, logits_stride=stride)
    out = {"counts": torch.full((S, E), -7, dtype=torch.int32, device=gpu), "rows": torch.full((S,), -7, dtype=torch.int32, device=gpu),
           "share": torch.full((S, E), NAN, device=gpu), "loss": torch.full((S,), NAN, device=gpu), "z": torch.full((S,), NAN, device=gpu)}
    if score == "sigmoid":
        del out["z"]
    if only:
        out = {n: out[n] for n in only}
    ws = torch.full((B.balance_workspace_bytes(s),), 0xFF, dtype=torch.uint8, device=gpu)
    B.balance(s, None if only == ["counts"] else l, ids, ws, seq_offsets=off, **out)
    return out


def on(gpu, *ts):
    return [None if t is None else t.to(gpu) for t in ts]


def check_forward(l, ids, off, gpu, score="softmax", S=1, tol=SUM):
    out = {k: v.cpu().numpy() for k, v in forward(*on(gpu, l, ids, off), gpu, score, S).items()}
    ref = balance_ref(l.double().numpy(), ids.numpy(), None if off is None else off.numpy(), score)
    assert np.array_equal(out["counts"], ref["counts"]) and np.array_equal(out["rows"], ref["rows"])
    for name in ("share", "loss", "z"):
        if name in out:
            assert np.array_equal(np.isnan(out[name]), np.isnan(ref[name])), name
            with np.errstate(over="ignore"):  # FP32's range ends below the square of its lowest value
                beyond = np.isinf(ref[name].astype(np.float32))
            assert np.isinf(out[name][beyond]).all(), name
            fine = ~np.isnan(ref[name]) & ~beyond
            # a log-sum-exp near 0 keeps what the largest logit and the logarithm lose: 2^-22 of values up to 8, squared
            assert (np.abs(out[name] - ref[name])[fine] <= tol * np.abs(ref[name])[fine] + (2.0 ** -36 if name == "z" else 2.0 ** -140)).all(), name
    return ref


SIZES = [(1, 1, 1), (1, 8, 8), (3, 5, 2), (16, 32, 4), (17, 33, 7), (64, 64, 8), (70, 65, 64), (130, 128, 1), (33, 129, 5), (300, 256, 8),
         (100, 257, 6), (40, 384, 6), (9, 512, 16), (8, 513, 3), (5, 1000, 33), (20, 1024, 64), (1025, 16, 2), (9000, 12, 3)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_forward_sizes(gpu, T, E, k, dtype, score):
    print(f"balance {T} x {E} top {k} {dtype} {score}", flush=True)
    for hole, S in ((0.0, 1), (0.2, 5)):
        l, ids, off = inputs(T, E, k, T + E, dtype, hole, S)
        check_forward(l, ids, off, gpu, score, S)


OFFSETS = {"empty ends": [0, 0, 0, 40, 40, 90, 90, 90], "gaps": [5, 17, 18, 19, 35, 36, 60, 77], "one row each": list(range(8)),
           "out of range": [-5, 3, 20, 64, 80, 91, 200, 1 << 40], "none": [90] * 8, "at the start": [0] * 8, "tiles": [0, 16, 32, 48, 64, 80, 88, 90],
           "behind": [-9, -8, -7, -6, -5, -4, -3, -2]}


@pytest.mark.parametrize("name", list(OFFSETS))
def test_forward_offsets(gpu, name):
    print(name, flush=True)
    for score in ("softmax", "sigmoid"):
        l, ids, _ = inputs(90, 20, 3, 4, F32, 0.2)
        check_forward(l, ids, torch.tensor(OFFSETS[name]), gpu, score, 7)


def test_forward_many_short_sequences(gpu):
    l, ids, _ = inputs(700, 24, 2, 5, F32, 0.1)
    check_forward(l, ids, torch.arange(1401).div(2, rounding_mode="floor"), gpu, S=1400)


# sequences within tiles of 16 rows (64 of 20000), over their borders, at them, and fewer, as many or more than there are tiles
TILED = {"borders": [0, 16, 32, 48, 64, 128, 256, 599, 600], "around borders": [0, 15, 17, 31, 32, 33, 47, 65, 300, 303, 600],
         "long ones between short": [0, 1, 2, 100, 101, 102, 103, 400, 401, 400 + 16, 580], "gaps": [20, 21, 90, 580, 581],
         "more than tiles": sorted([*range(0, 600, 7), *([300] * 10)]), "as many": [*range(0, 590, 16)] + [600],
         "one of all between empty ones": [0] * 30 + [600] * 30, "rows behind": [*range(0, 100)], "none": [600] * 50}


@pytest.mark.parametrize("name", list(TILED))
def test_forward_tiles(gpu, name):
    print(name, flush=True)
    l, ids, _ = inputs(600, 36, 3, 4, F32, 0.1)
    check_forward(l, ids, torch.tensor(TILED[name]), gpu, S=len(TILED[name]) - 1)


@pytest.mark.parametrize("T,E,S", [(256, 40, 1), (256, 40, 400), (257, 40, 1), (257, 40, 2), (1024, 33, 7), (1024, 33, 8), (1025, 33, 64),
                                   (1025, 33, 65), (1025, 33, 66), (1500, 48, 1300), (20000, 16, 312), (20000, 16, 313), (20000, 16, 4000)])
def test_forward_sequences_by_tiles(gpu, T, E, S):
    print(T, E, S, flush=True)
    l, ids, off = inputs(T, E, 2, T + S, F32, 0.1, S)
    check_forward(l, ids, off, gpu, S=S)


def test_forward_falling_offsets_stay_in_bounds(gpu):
    """Their result is not specified; the call ends, and leaves what it was not given alone."""
    l, ids, _ = inputs(300, 20, 3, 4)
    forward(*on(gpu, l, ids, torch.tensor([200, 10, 280, -4, 1 << 50, 7, 90, 3])), gpu, S=7)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E,stride,at", [(20, 24, 0), (20, 23, 0), (64, 100, 4), (64, 100, 1), (33, 40, 3), (1024, 1028, 2)])
def test_strided_rows(gpu, E, stride, at, dtype):
    wide = torch.full((50, stride + 8), 3e4, dtype=dtype)
    l, ids, _ = inputs(50, E, 4, 6, dtype, 0.1)
    wide.view(-1)[at:at + 50 * stride].view(50, stride)[:, :E] = l
    g = wide.to(gpu).view(-1)[at:at + 50 * stride].view(50, stride)[:, :E]
    a = forward(g, ids.to(gpu), None, gpu, stride=stride)
    b = forward(*on(gpu, l, ids, None), gpu)
    for n in ("counts", "rows"):
        assert torch.equal(a[n], b[n])
    assert torch.allclose(a["share"], b["share"], rtol=SUM, atol=0)
    d = [gradient(x, ids.to(gpu), None, gpu, st, counts=b["counts"], rows=b["rows"], d_loss=torch.ones(1, device=gpu),
                  d_topk_w=torch.ones(50, 4, device=gpu)) for x, st in ((g, stride), (l.to(gpu), 0))]
    assert torch.allclose(d[0].float(), d[1].float(), rtol=2.0 ** -7 if dtype == BF16 else 2.0 ** -12, atol=2.0 ** -24)


def test_forward_each_output_alone(gpu):
    l, ids, off = on(gpu, *inputs(200, 48, 4, 7, F32, 0.1, 3))
    whole = forward(l, ids, off, gpu, S=3)
    for n in whole:
        assert torch.equal(forward(l, ids, off, gpu, S=3, only=[n])[n], whole[n]), n


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_forward_is_the_same_every_time(gpu, score):
    l, ids, off = on(gpu, *inputs(5000, 100, 6, 8, F32, 0.1, 9))
    a = forward(l, ids, off, gpu, score, 9)
    for _ in range(5):
        b = forward(l, ids, off, gpu, score, 9)
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_no_rows(gpu):
    for S, off in ((1, None), (3, torch.tensor([0, 0, 5, 5], device=gpu))):
        l, ids = torch.empty(0, 20, device=gpu), torch.empty(0, 3, dtype=torch.int64, device=gpu)
        out = forward(l, ids, off, gpu, S=S)
        assert all((v == 0).all() for v in out.values())
        gradient(l, ids, off, gpu, S=S, counts=out["counts"], rows=out["rows"], d_loss=torch.ones(S, device=gpu))


def test_ids_outside_are_not_counted(gpu):
    l, ids, _ = inputs(40, 10, 3, 9)
    ids[3, 1], ids[4, 0], ids[5, 2], ids[6, 0] = 10, -1, 1 << 40, -(1 << 62)
    ids[7, 1] = ids[7, 0]
    ref = check_forward(l, ids, None, gpu)
    assert ref["counts"].sum() == 116


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_odd_logits(gpu, score):
    """Masks of the type's lowest value, infinities and NaN, very small scores."""
    l, ids, _ = inputs(12, 40, 4, 10)
    l[1] = torch.finfo(F32).min
    l[2, 3:] = torch.finfo(F32).min
    l[3], l[4] = -300.0 + l[3], 200.0 + l[4]
    l[5] = -INF
    l[6, 1:] = -INF
    off = torch.arange(13)
    check_forward(l, ids, off, gpu, score, 12)
    l[7, 3], l[8, 3] = NAN, INF
    l[9] = -INF
    l[9, 4] = NAN
    o = forward(*on(gpu, l, ids, off), gpu, score, 12)
    bad = [7, 9] + ([8] if score == "softmax" else [])
    for r in range(12):
        assert bool(torch.isnan(o["share"][r]).all()) == (r in bad), r
    assert o["rows"].cpu().tolist() == [1] * 5 + [0] + [1] * 6
    if score == "sigmoid":
        assert o["share"][8, 3] > 0.01


# ---- gradient

def gradient(l, ids, off, gpu, stride=0, S=1, score="softmax", renormalize=True, scale=1.0, out=None, **kw):
    T, E = l.shape
    s = B.make_balance(T, E, ids.shape[1], num_seqs=S, score=score, logits_dtype=l.dtype, logits_stride=stride,
                       renormalize=renormalize, scale=scale)
    out = torch.full((T, E), 7.0, dtype=l.dtype, device=gpu) if out is None else out
    B.gate_grad(s, l, ids, out, seq_offsets=off, **kw)
    return out


def magnitudes(l, ids, counts, rows, off, score, renorm, scale, d_loss, d_z, d_topk_w):
    """The sum of the magnitudes of what a gradient's element is the sum of."""
    T, E = l.shape
    m = np.zeros((T, E))
    for s, (a, b) in enumerate(spans(T, off)):
        g = np.zeros(E)
        if d_loss is not None and rows[s] and counts[s].sum():
            # the difference to an even load, which is what is computed
            g = np.abs(d_loss[s] * (E * counts[s] / counts[s].sum() - 1.0) / rows[s])
        for t in range(a, b):
            p, lse, _ = row_shares(l[t], score)
            m[t] = p * (g + p @ g)
            if d_z is not None and rows[s]:
                m[t] += p * 2 * abs(d_z[s]) * (abs(lse) + 1) / rows[s]
            if d_topk_w is not None:
                ok = [(j, int(e)) for j, e in enumerate(ids[t]) if 0 <= e < E and not np.isneginf(l[t, e])]
                if ok:
                    e, d = np.array([x for _, x in ok]), np.abs(scale * d_topk_w[t])[[j for j, _ in ok]]
                    sc = row_scores(l[t], score)[0][e]
                    if renorm:
                        sc = row_shares(l[t][e], score)[0]
                    np.add.at(m[t], e, sc * (d + (sc @ d if renorm else 0)))
                    if score == "softmax" and not renorm:
                        m[t] += p * (sc @ d)
    return m


def check_gradient(l, ids, off, gpu, score="softmax", renorm=True, scale=1.0, S=1, parts=("loss", "z", "w"), seed=0):
    g = np.random.default_rng(seed)
    T, E = l.shape
    o = None if off is None else off.numpy()
    fw = balance_ref(l.double().numpy(), ids.numpy(), o, "softmax")
    kw = {}
    if "loss" in parts:
        kw["d_loss"] = torch.from_numpy(g.normal(size=S)).float()
    if "z" in parts and score == "softmax":
        kw["d_z"] = torch.from_numpy(g.normal(size=S)).float()
    if "w" in parts:
        kw["d_topk_w"] = torch.from_numpy(g.normal(size=tuple(ids.shape)) / T).float()
    dev = {n: v.to(gpu) for n, v in kw.items()}
    if "d_loss" in kw:
        dev["counts"] = torch.from_numpy(fw["counts"]).int().to(gpu)
    if "d_loss" in kw or "d_z" in kw:
        dev["rows"] = torch.from_numpy(fw["rows"]).int().to(gpu)
    got = gradient(*on(gpu, l, ids, off), gpu, S=S, score=score, renormalize=renorm, scale=scale, **dev).double().cpu().numpy()
    ln = l.double().numpy()
    num = {n: v.double().numpy() for n, v in kw.items()}
    ref = gate_grad_ref(ln, ids.numpy(), fw["counts"], fw["rows"], offsets=o, score=score, renormalize=renorm, scale=scale, **num)
    mag = magnitudes(ln, ids.numpy(), fw["counts"], fw["rows"], o, score, renorm, scale, *(num.get(n) for n in ("d_loss", "d_z", "d_topk_w")))
    outside = np.isnan(ref)
    assert (got[outside] == 7).all()  # rows in no sequence are left as they were
    ref, got, mag = ref[~outside], got[~outside], mag[~outside]
    tol = (2.0 ** -17) * mag + 2.0 ** -130
    if l.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    assert (np.abs(got - ref) <= tol).all(), f"{(np.abs(got - ref) / np.maximum(tol, 1e-300)).max():.3g} times the bound"


@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", SIZES[:-1])
def test_gradient_sizes(gpu, T, E, k, dtype, score, renorm):
    print(f"grad {T} x {E} top {k} {dtype} {score} {renorm}", flush=True)
    for hole, S in ((0.0, 1), (0.2, 5)):
        l, ids, off = inputs(T, E, k, T + E + 1, dtype, hole, S)
        check_gradient(l, ids, off, gpu, score, renorm, 2.5, S)


@pytest.mark.parametrize("parts", [("loss",), ("z",), ("w",), ("loss", "w"), ("z", "w")])
@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_gradient_parts(gpu, parts, score, renorm):
    if parts == ("z",) and score == "sigmoid":
        return
    l, ids, off = inputs(120, 40, 5, 3, F32, 0.1, 4)
    check_gradient(l, ids, off, gpu, score, renorm, -1.5, 4, parts)


@pytest.mark.parametrize("name", list(OFFSETS))
def test_gradient_offsets(gpu, name):
    for score in ("softmax", "sigmoid"):
        l, ids, _ = inputs(90, 20, 3, 4, F32, 0.2)
        check_gradient(l, ids, torch.tensor(OFFSETS[name]), gpu, score, True, 1.0, 7)


@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_gradient_odd_ids(gpu, score, renorm):
    """An id twice, ids that are none, ids whose logit is masked, a row without any."""
    l, ids, _ = inputs(30, 24, 6, 5)
    ids[3, 1] = ids[3, 0]
    ids[4, :] = ids[4, 0]
    ids[5, 2], ids[6, 0], ids[7, 5] = 24, -1, 1 << 40
    ids[8] = -1
    l[9, ids[9, 1]] = -INF
    l[10, ids[10]] = -INF
    l[11] = -INF
    check_gradient(l, ids, None, gpu, score, renorm, 1.0)


@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_gradient_far_logits(gpu, score, renorm):
    l, ids, _ = inputs(20, 40, 4, 6)
    l[0:4] -= 60.0
    l[4:8] += 60.0
    l[8:12, ::2] -= 50.0
    ids[10] = torch.arange(4) * 2
    l[12] = torch.finfo(F32).min
    check_gradient(l, ids, None, gpu, score, renorm, 1.0)


def test_gradient_of_an_even_load_is_zero(gpu):
    l, ids, _ = inputs(64, 16, 1, 7)
    out = gradient(*on(gpu, l, ids, None), gpu, counts=torch.full((1, 16), 4, dtype=torch.int32, device=gpu),
                   rows=torch.tensor([64], dtype=torch.int32, device=gpu), d_loss=torch.ones(1, device=gpu))
    assert (out == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_nan_stays_in_its_row(gpu, score):
    l, ids, _ = inputs(10, 20, 3, 8)
    l[4, 7], l[4, 8] = NAN, -INF
    fw = forward(*on(gpu, inputs(10, 20, 3, 8)[0], ids, None), gpu, score)
    out = gradient(*on(gpu, l, ids, None), gpu, score=score, counts=fw["counts"], rows=fw["rows"], d_loss=torch.ones(1, device=gpu),
                   d_topk_w=torch.ones(10, 3, device=gpu))
    nan = torch.isnan(out)
    assert nan[4].sum() == 19 and out[4, 8] == 0 and not nan[torch.arange(10) != 4].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [48, 33, 384])
def test_gradient_in_place(gpu, E, dtype):
    l, ids, off = on(gpu, *inputs(333, E, 6, 9, dtype, 0.1, 4))
    fw = forward(l, ids, off, gpu, S=4)
    kw = dict(S=4, counts=fw["counts"], rows=fw["rows"], d_loss=torch.ones(4, device=gpu), d_topk_w=torch.randn(333, 6, device=gpu))
    inside = torch.zeros(333, dtype=torch.bool, device=gpu)
    inside[int(off[0]):int(off[-1])] = True
    a, x = gradient(l, ids, off, gpu, **kw), l.clone()
    gradient(x, ids, off, gpu, out=x, **kw)
    assert torch.equal(x[inside], a[inside]) and torch.equal(x[~inside], l[~inside])


def test_gradient_of_summed_counts(gpu):
    """Counts of several ranks, added up: past 2^31 / E."""
    l, ids, _ = inputs(50, 32, 4, 11)
    counts = torch.randint(1 << 26, 1 << 27, (1, 32), generator=torch.Generator().manual_seed(0), dtype=torch.int32)
    ref = gate_grad_ref(l.double().numpy(), ids.numpy(), counts.numpy(), [50], d_loss=[1.0])
    got = gradient(*on(gpu, l, ids, None), gpu, counts=counts.to(gpu), rows=torch.tensor([50], dtype=torch.int32, device=gpu),
                   d_loss=torch.ones(1, device=gpu)).double().cpu().numpy()
    m = magnitudes(l.double().numpy(), ids.numpy(), counts.numpy(), [50], None, "softmax", True, 1.0, np.ones(1), None, None)
    assert (np.abs(got - ref) <= 2.0 ** -17 * m).all()
