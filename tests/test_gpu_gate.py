"""GPU parity of moe_gate: ids equal to the float64 oracle's, weights within their roundings.

Weights come from scores in 64 bits and are rounded once: 2^-24, and as much again for the exponentials'
and the sum's own 64-bit error.  Softmax weights that are not renormalised are divided by a 64-bit sum of the
whole row's exponentials in 32 bits: 10 * 2^-24 relative (the argument's rounding, weighted, at most ln(1024) < 7
times 2^-24, the exponential 3 * 2^-24), with the weight's own rounding below 2^-20 (test_gate_whole_row_sums);
the tests of other things allow 2^-19.
"""
import itertools

import numpy as np
import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B
from oracle.front import gate_ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def run(logits, k, bias=None, shape=None, **kw):
    T, E = logits.shape
    s = shape or B.make_gate(T, E, k, logits_dtype=logits.dtype, **kw)
    ids = torch.full((T, k), 777, dtype=torch.int64, device=logits.device)
    w = torch.full((T, k), NAN, device=logits.device)
    B.gate(s, logits, ids, w, bias=bias)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.double().cpu().numpy()


def check(logits, k, bias=None, **kw):
    ids, w = run(logits, k, bias, **kw)
    rids, rw = gate_ref(logits.double().cpu().numpy(), k, bias=None if bias is None else bias.cpu().numpy(), **kw)
    assert np.array_equal(ids, rids)
    whole_row = kw.get("score", "softmax") == "softmax" and not kw.get("renormalize", True)
    tol = 2.0 ** -19 if whole_row else 2.0 ** -23
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    fine = ~np.isnan(rw)
    assert (np.abs(w - rw)[fine] <= tol * np.abs(rw)[fine] + 2.0 ** -140).all()


def normal(T, E, seed, gpu, dtype=F32, scale=1.0):
    return (torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(gpu)


def balance(E, seed, gpu):
    return torch.randint(-100, 101, (E,), generator=torch.Generator().manual_seed(seed)).float().to(gpu) * 1e-3


SIZES = [(1, 1, 1), (3, 2, 1), (2, 8, 2), (70, 8, 8), (5, 63, 6), (9, 64, 8), (9, 65, 8), (33, 100, 7), (130, 128, 64),
         (4, 255, 8), (300, 256, 8), (7, 257, 1), (100, 384, 6), (3, 511, 12), (20, 512, 8), (3, 513, 5), (6, 1000, 33),
         (5, 1024, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gate_sizes(gpu, T, E, k, dtype):
    print(f"gate T={T} E={E} k={k} {dtype}", flush=True)
    l = normal(T, E, T + E, gpu, dtype)
    for score, renorm in itertools.product(["softmax", "sigmoid"], [True, False]):
        check(l, k, score=score, renormalize=renorm, scale=2.5)
        check(l, k, balance(E, 1, gpu), score=score, renormalize=renorm)


GROUPS = [(32, 4, 2, 4), (256, 8, 4, 8), (256, 8, 1, 8), (64, 64, 5, 5), (60, 4, 3, 8), (120, 8, 2, 16), (384, 8, 3, 6),
          (1024, 16, 4, 64), (1008, 63, 7, 10), (96, 2, 2, 4), (20, 5, 5, 20), (7, 7, 2, 1)]


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,groups,kept,k", GROUPS)
def test_gate_groups(gpu, E, groups, kept, k, group_score):
    print(f"gate E={E} groups={groups} kept={kept} k={k} {group_score}", flush=True)
    for score, biased, dtype in itertools.product(["softmax", "sigmoid"], [True, False], [F32, BF16]):
        l = normal(60, E, E + kept, gpu, dtype)
        check(l, k, balance(E, 2, gpu) if biased else None, score=score, num_groups=groups, topk_groups=kept,
              group_score=group_score)


@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_ties(gpu, score, biased, groups, kept):
    """Few distinct logits and biases: most choices are ties, of experts and of groups, -0 and +0 among them."""
    g = torch.Generator().manual_seed(3)
    l = torch.randint(-2, 3, (200, 64), generator=g).float() * torch.where(torch.rand(200, 64, generator=g) < 0.5, 1, -1)
    b = (torch.randint(0, 2, (64,), generator=g).float() * 0.25).to(gpu) if biased else None
    for dtype, gs in itertools.product([F32, BF16], ["max", "top2"]):
        check(l.to(dtype).to(gpu), 8, b, score=score, num_groups=groups, topk_groups=kept, group_score=gs)
    check(torch.zeros(3, 64, device=gpu), 8, b, score=score, num_groups=groups, topk_groups=kept)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_near_ties(gpu, score):
    """Orders that 32 bits would get wrong: sums of score and bias a few 2^-26 apart."""
    g = torch.Generator().manual_seed(4)
    T, E = 300, 64
    l = torch.randn(T, E, generator=g) * 0.2
    s = torch.sigmoid(l.double()) if score == "sigmoid" else torch.softmax(l.double(), -1)
    bias = (1.0 - s[0]).float()
    l[1:] = l[0] + torch.randint(-3, 4, (T - 1, E), generator=g) * 2.0 ** -26
    l[150:] = l[0] + torch.randint(-1, 2, (150, E), generator=g) * 2.0 ** -23
    for groups, kept in ((1, 1), (8, 4)):
        for gs in ("max", "top2"):
            check(l.to(gpu), 8, bias.to(gpu), score=score, num_groups=groups, topk_groups=kept, group_score=gs)
            check(l.to(gpu), 8, score=score, num_groups=groups, topk_groups=kept, group_score=gs)


@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2), (32, 8)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_masks(gpu, score, biased, groups, kept):
    """Rows from all experts down to none; experts masked by logit or by bias; groups masked whole."""
    T, E, k = 65, 64, 8
    l = normal(T, E, 5, gpu)
    order = torch.rand(T, E, generator=torch.Generator().manual_seed(6)).argsort(1).to(gpu)
    l[order < torch.arange(T, device=gpu)[:, None]] = -INF         # row t masks t experts; the last row all 64
    l[3, 16:] = -INF
    b = None
    if biased:
        b = balance(E, 7, gpu)
        b[5], b[17], b[32:48] = -INF, -INF, -INF
    for renorm, gs in itertools.product([True, False], ["max", "top2"]):
        check(l, k, b, score=score, num_groups=groups, topk_groups=kept, group_score=gs, renormalize=renorm)
    ids, w = run(l, k, b, score=score)
    assert (ids[T - 1] == -1).all() and (w[T - 1] == 0).all()
    check(torch.full((5, E), -INF, device=gpu).to(BF16), k, b, score=score, num_groups=groups, topk_groups=kept)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_extreme_logits(gpu, score, biased):
    """Far apart, saturated and lowest-value logits; a sum of scores that is zero."""
    l = normal(40, 96, 8, gpu, scale=300.0)
    l[1] = torch.finfo(F32).min
    l[2] = -1e4 - torch.arange(96, device=gpu)
    l[3] = 1e4 + torch.arange(96, device=gpu)
    l[4, 1::2] = torch.finfo(F32).min
    l[5] = torch.arange(96, device=gpu) * 1e-42                     # subnormal
    b = balance(96, 9, gpu) if biased else None
    for renorm in (True, False):
        check(l, 8, b, score=score, renormalize=renorm)


@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_nan_and_infinity(gpu, score, groups, kept):
    l = normal(6, 64, 10, gpu)
    l[0, 40], l[1, 3], l[1, 50], l[2, 7] = NAN, NAN, NAN, INF
    l[3, 5:] = -INF
    l[3, 2] = NAN
    for gs in ("max", "top2"):
        for b in (None, balance(64, 11, gpu)):
            check(l, 6, b, score=score, num_groups=groups, topk_groups=kept, group_score=gs)
            check(l, 6, b, score=score, num_groups=groups, topk_groups=kept, group_score=gs, renormalize=False)


def test_gate_rows(gpu):
    """Strided rows at odd offsets, many rows, rows behind the last, and a scale of any sign."""
    l = normal(3000, 60, 12, gpu)
    want = run(l, 6)
    for dtype, off, stride in ((F32, 1, 77), (BF16, 3, 63)):
        wide = torch.full((3001, stride), INF, dtype=dtype, device=gpu)
        flat = wide.view(-1)[off:]
        rows = flat.as_strided((3000, 60), (stride, 1))
        rows.copy_(l)
        s = B.make_gate(3000, 60, 6, logits_dtype=dtype, logits_stride=stride)
        ids, w = run(rows, 6, shape=s)
        ref = run(l.to(dtype), 6)
        assert np.array_equal(ids, ref[0]) and np.array_equal(w, ref[1])
    ids = torch.full((10, 6), 9, dtype=torch.int64, device=gpu)
    w = torch.full((10, 6), 9.0, device=gpu)
    B.gate(B.make_gate(7, 60, 6), l[:7], ids[:7], w[:7])
    torch.cuda.synchronize()
    assert np.array_equal(ids[:7].cpu().numpy(), want[0][:7]) and (ids[7:] == 9).all() and (w[7:] == 9.0).all()
    check(l[:50], 6, scale=-0.5)
    check(l[:50], 6, scale=0.0)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(64, 4, 2), (256, 8, 3), (64, 16, 5), (512, 8, 4), (320, 32, 7), (96, 3, 1)])
def test_gate_groups_too_close_for_32_bits(gpu, E, groups, kept, score, biased):
    """Pairs whose sums of scores differ by less than FP32 tells, another expert of each group just below them."""
    g = torch.Generator().manual_seed(64)
    T, n = 60, E // groups
    l = torch.randn(T, groups, n, generator=g) * 0.3 - 3.0
    a = torch.rand(T, groups, generator=g).double() + 0.5
    if score == "sigmoid":      # s(a) + s(b) = 1.4
        b = torch.logit(1.4 - torch.sigmoid(a))
    else:                       # e^a + e^b = 6
        b = torch.log(6.0 - torch.exp(a))
    l[..., 0], l[..., n // 2], l[..., n - 1] = a.float(), b.float(), b.float() - 2.0 ** -21
    l = l.reshape(T, E).to(gpu)
    bias = torch.full((E,), 0.25, device=gpu) if biased else None
    for group_score in ("top2", "max"):
        check(l, min(4, n * kept), bias=bias, score=score, num_groups=groups, topk_groups=kept, group_score=group_score)
    same = l[:1].repeat(T, 1).view(T, groups, n)    # all groups alike: the lowest are kept
    same[1:] = same[1:, :1]
    check(same.reshape(T, E), min(4, n * kept), bias=bias, score=score, num_groups=groups, topk_groups=kept, group_score="top2")


@pytest.mark.parametrize("part", [1.0, 0.5, 0.999])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_bias_cancels_scores(gpu, score, part):
    """A bias that takes back the scores of the first row: order values that differ by the bias's rounding only,
    where scores differ by all of their own."""
    E = 128
    l = normal(40, E, 63, gpu)
    l[1:20] = l[0]
    l[5, :64] += 2.0 ** -20
    d = l[0].double()
    s = torch.softmax(d, 0) if score == "softmax" else torch.sigmoid(d)
    check(l, 8, bias=(-s * part).float(), score=score)
    check(l, 8, bias=(s.mean() - s * part).float(), score=score, num_groups=4, topk_groups=2, group_score="top2")


@pytest.mark.parametrize("groups,kept,group_score", [(1, 1, "max"), (8, 4, "max"), (8, 4, "top2")])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_bias_without_bounds(gpu, score, groups, kept, group_score):
    """Biases that are not finite, or that leave no room between the scores."""
    E, big = 64, torch.finfo(F32).max
    l = normal(9, E, 60, gpu)
    l[2, 5::7], l[3] = -INF, -INF
    for values in ({3: NAN, 40: NAN}, {7: INF}, {7: INF, 8: INF, 50: -INF}, {e: -INF for e in range(E) if e % 9},
                   {1: big, 2: -big}, {e: -big for e in range(E)}, {e: big for e in range(E)}, {5: NAN, 6: INF, 7: -INF}):
        bias = balance(E, 61, gpu)
        for e, v in values.items():
            bias[e] = v
        check(l, 6, bias=bias, score=score, num_groups=groups, topk_groups=kept, group_score=group_score)


def test_gate_more_rows_than_a_grid_axis(gpu):
    """Over 2^24 rows of two experts; the larger sigmoid, rounded twice at most (64 bits, then 32)."""
    T = (1 << 24) + 9
    g = torch.Generator(device=gpu).manual_seed(62)
    l = torch.randn(T, 2, generator=g, device=gpu)
    ids = torch.full((T, 1), 777, dtype=torch.int64, device=gpu)
    w = torch.full((T, 1), NAN, device=gpu)
    B.gate(B.make_gate(T, 2, 1, score="sigmoid", renormalize=False), l, ids, w)
    torch.cuda.synchronize()
    assert torch.equal(ids[:, 0], (l[:, 1] > l[:, 0]).long())
    want = torch.sigmoid(l.max(dim=1).values.double())
    assert ((w[:, 0].double() - want).abs() <= 2.0 ** -23 * want).all()


def test_gate_no_tokens(gpu):
    e = torch.zeros(0, 8, device=gpu)
    B.gate(B.make_gate(0, 8, 2), e, torch.zeros(0, 2, dtype=torch.int64, device=gpu), torch.zeros(0, 2, device=gpu))


def test_gate_binding_refusals(gpu):
    l, s = normal(4, 16, 13, gpu), B.make_gate(4, 16, 2)
    ids, w = torch.empty(4, 2, dtype=torch.int64, device=gpu), torch.empty(4, 2, device=gpu)
    for a, kw in (((l[:3], ids, w), {}), ((l.to(BF16), ids, w), {}), ((l, ids.int(), w), {}), ((l, ids, w.double()), {}),
                  ((l, ids[:3], w), {}), ((l, ids, w), dict(bias=torch.zeros(15, device=gpu))),
                  ((l, ids, w), dict(bias=torch.zeros(16))), ((l, ids, w), dict(bias=torch.zeros(16, device=gpu).to(BF16)))):
        with pytest.raises((TypeError, ValueError)):
            B.gate(s, *a, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E,k,score,biased", [(256, 8, "sigmoid", True), (256, 8, "softmax", True), (384, 6, "sigmoid", False),
                                              (100, 14, "sigmoid", True), (24, 5, "softmax", True), (520, 9, "sigmoid", True)])
def test_gate_many_rows(gpu, E, k, score, biased, dtype):
    """Enough rows that near ties of every kind occur, against a stable sort in 64 bits."""
    T = 60000
    l = normal(T, E, 21, gpu, dtype)
    b = balance(E, 22, gpu) if biased else None
    ids, _ = run(l, k, b, score=score)
    d = l.double()
    s = torch.softmax(d, -1) if score == "softmax" else 1 / (1 + torch.exp(-d))
    c = s + b.double() if biased else d
    want = torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :k].cpu().numpy()
    assert np.array_equal(ids, want)


@pytest.mark.parametrize("groups,kept,group_score", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 100, 1024])
def test_gate_biases_far_below_zero(gpu, E, score, groups, kept, group_score):
    """Candidates whose biases are all far below zero, the best ones last: FP32 has no room for steps of 2^-22 there,
    and sums of two of the lowest are beyond its range."""
    print(f"gate E={E} {score} groups={groups} {group_score}", flush=True)
    l = normal(5, E, 70, gpu)
    l[2, 3::5], l[3] = -INF, -INF
    rise = torch.arange(E, device=gpu, dtype=torch.float64) / E
    for low, high in ((-1e9, -9e8), (-2e29, -1e29), (-2.0 ** 100, -2.0 ** 100 * (1 - 2.0 ** -13)), (-2e32, -1.4e32),
                      (-3.4e38, -3.3e38), (-3.4e38, -1.0)):
        check(l, 6, bias=(low + (high - low) * rise).float(), score=score, num_groups=groups, topk_groups=kept,
              group_score=group_score)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(3, 1, 1), (33, 1, 1), (100, 1, 1), (257, 1, 1), (513, 1, 1), (60, 3, 2), (1008, 63, 7)])
def test_gate_rows_without_candidates(gpu, E, groups, kept, score, dtype):
    """Sizes at which lanes hold places past the row's end, in rows that leave no candidate, the last ones of their
    memory: masked by the logits, by the bias, or by both; one candidate between them."""
    print(f"gate E={E} groups={groups} {score} {dtype}", flush=True)
    k = min(8, E // groups * kept)
    l = normal(21, E, 71, gpu, dtype)
    l[::2] = -INF
    l[16, E - 1] = 0.5
    half = balance(E, 72, gpu)
    half[E // 2:] = -INF
    l[19, :E // 2] = -INF
    for bias in (torch.full((E,), -INF, device=gpu), half, balance(E, 73, gpu)):
        for group_score in ("max", "top2"):
            check(l, k, bias=bias, score=score, num_groups=groups, topk_groups=kept, group_score=group_score)
    ids, w = run(l, k, half, score=score, num_groups=groups, topk_groups=kept)
    assert (ids[[0, 19, 20]] == -1).all() and (w[[0, 19, 20]] == 0).all()


# (lanes of a row, experts of a lane, keys it keeps) of every kernel, and shapes that it takes: E, groups, kept, k; the
# second of each in lanes that hold no runs of 4
KERNELS = {(16, 4, 4): [(64, 1, 1, 8), (45, 3, 2, 16)], (16, 8, 8): [(128, 4, 2, 8), (63, 9, 5, 16)],
           (16, 16, 8): [(256, 8, 3, 8), (135, 9, 4, 5)], (16, 16, 16): [(256, 8, 3, 16), (135, 9, 4, 9)],
           (16, 24, 8): [(384, 8, 3, 8), (331, 1, 1, 7)], (16, 32, 8): [(512, 16, 5, 8), (465, 15, 4, 8)],
           (16, 32, 16): [(512, 16, 5, 12), (465, 15, 4, 16)], (64, 16, 8): [(1024, 1, 1, 8), (1001, 1, 1, 3)],
           (64, 16, 16): [(1024, 16, 4, 16), (806, 13, 3, 9)],
           (64, 32, 8): [(960, 5, 3, 8), (1023, 3, 2, 8), (1001, 7, 3, 8), (1023, 33, 9, 8)],
           (64, 32, 16): [(960, 5, 3, 16), (1020, 6, 4, 12), (1023, 3, 2, 12), (561, 17, 5, 16)],
           (64, 0, 0): [(128, 4, 2, 17), (1023, 3, 2, 64)]}


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("kernel,shape", [(k, s) for k, v in KERNELS.items() for s in v])
def test_gate_every_kernel(gpu, kernel, shape, group_score):
    """Random rows, rows of near ties, masked rows, in both types, with and without a bias."""
    E, groups, kept, k = shape
    print(f"gate {kernel} E={E} groups={groups} kept={kept} k={k} {group_score}", flush=True)
    assert B.gate_lanes(B.make_gate(1, E, k, num_groups=groups, topk_groups=kept)) == kernel
    g = torch.Generator().manual_seed(E + k)
    l = torch.randn(36, E, generator=g)
    near = torch.randn(E, generator=g) * 0.2
    l[12:18] = near + torch.randint(-2, 3, (6, E), generator=g) * 2.0 ** -24
    l[18:24] = torch.randint(-3, 4, (6, E), generator=g).float()
    l[24:34][torch.rand(10, E, generator=g) < torch.linspace(0.1, 0.99, 10)[:, None]] = -INF
    l[34] = -INF
    l[35, E - 1] = 9.0
    bias = (1.0 - torch.sigmoid(near)).to(gpu)
    for dtype, b, score in itertools.product([F32, BF16], [None, bias, balance(E, 74, gpu)], ["softmax", "sigmoid"]):
        check(l.to(dtype).to(gpu), k, bias=b, score=score, num_groups=groups, topk_groups=kept, group_score=group_score)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E,k,groups,kept", [(64, 8, 1, 1), (256, 8, 8, 4), (384, 6, 1, 1), (1024, 16, 1, 1), (96, 24, 1, 1)])
def test_gate_whole_row_sums(gpu, E, k, groups, kept, dtype):
    """Softmax weights over the whole row's sum: 10 units of 2^-24 of the sum and 1 of the weight, products of them
    and 64-bit roundings below a tenth of a unit."""
    for i, scale in enumerate((0.01, 1.0, 4.0, 30.0)):
        l = normal(200, E, 80 + i, gpu, dtype, scale)
        l[100:][torch.rand(100, E, generator=torch.Generator().manual_seed(i)).to(gpu) < 0.3] = -INF
        for bias in (None, balance(E, 90, gpu)):
            kw = dict(num_groups=groups, topk_groups=kept, renormalize=False)
            ids, w = run(l, k, bias, **kw)
            rids, rw = gate_ref(l.double().cpu().numpy(), k, bias=None if bias is None else bias.cpu().numpy(), **kw)
            assert np.array_equal(ids, rids)
            assert (np.abs(w - rw) <= 11.1 * 2.0 ** -24 * rw + 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,k", [(28, 4, 3, 1), (64, 8, 3, 6), (48, 8, 1, 2), (1008, 63, 7, 10), (256, 8, 7, 16)])
def test_gate_group_marks_beyond_fp32(gpu, E, groups, kept, k, score, dtype):
    """Groups whose two best sum below FP32's lowest value, next to groups without candidates, which come first."""
    print(f"gate E={E} groups={groups} kept={kept} {score} {dtype}", flush=True)
    n = E // groups
    l = normal(40, E, 75, gpu, dtype)
    for t in range(40):                                # from no empty group to all but one
        l[t, :n * (t % groups)] = -INF
    g = torch.Generator().manual_seed(76)
    for low, high in ((-3.4e38, -3.0e38), (-3.0e38, -3.0e38), (-1.8e38, -1.6e38)):
        bias = (torch.rand(E, generator=g) * (high - low) + low).to(gpu)
        check(l, k, bias=bias, score=score, num_groups=groups, topk_groups=kept, group_score="top2")
        bias[n // 2::n + 1] = 0.25                     # a few groups with one usual expert
        check(l, k, bias=bias, score=score, num_groups=groups, topk_groups=kept, group_score="top2")
