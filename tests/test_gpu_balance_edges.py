"""moe_balance and moe_gate_grad where they can go wrong.  Tolerances as derived in test_gpu_balance.py."""
import itertools

import numpy as np
import pytest
import torch

from test_gpu_balance import INF, NAN, check_forward, check_gradient, forward, gradient, inputs, on

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ---- more sequences than the lanes that the last rows fill

@pytest.mark.parametrize("behind", [0, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,S", [(1001, 64, 20), (1003, 33, 9), (9, 8, 30), (1, 8, 30), (1001, 128, 40), (7, 100, 200), (1001, 256, 50),
                                   (65, 384, 64), (101, 20, 101), (1025, 64, 1000), (9001, 16, 6000)])
def test_gradient_last_rows_of_many_sequences(gpu, T, E, S, score, behind):
    """Sequences of equal length, empty ones among them where there are more than rows; `behind`: rows that follow the last."""
    print(f"grad {T} x {E} in {S}", flush=True)
    end = max(T - behind, 0)
    off = torch.from_numpy(np.linspace(0, end, S + 1).round().astype(np.int64))
    l, ids, _ = inputs(T, E, 3, T + S, F32, 0.1)
    for seed in range(2):
        check_gradient(l, ids, off, gpu, score, True, 1.0, S, seed=seed)


# ---- renormalised weights that are formed again, over the largest of the chosen

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E,k", [(8, 1), (20, 3), (32, 9), (64, 2), (64, 11), (100, 3), (128, 20), (256, 8), (256, 40), (300, 6), (384, 33),
                                 (512, 5), (1000, 8), (1024, 64)])
def test_gradient_of_chosen_far_below_the_others(gpu, E, k, dtype, score):
    """As with a bias that outweighs the scores: the chosen experts' scores are below 2^-126 of the others'."""
    l, _, _ = inputs(33, E, k, E + k, dtype)
    g = torch.Generator().manual_seed(E)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(33)])
    low = -128.0 - torch.randint(0, 4, (33, k), generator=g).to(dtype)
    check_gradient(l.scatter(1, ids, low), ids, None, gpu, score, True, 1.0, 1, ("w",))


# ---- logits of any size

def far_rows(seed, E=24):
    """Rows around tops of any power of two, both signs: neighbours within two steps of FP32 (and of 1), whose distance is
    exact and either at most 16 or above 127, where exponentials count as 0."""
    g = np.random.default_rng(seed)
    rows = []
    for e in [0, 10, 16, 19, 20, 21, 24, 26, *range(31, 64, 2), 75, 90, 98, 99, 100, 101, 120, 126]:
        for sign in (1, -1):
            top = np.float32(sign * g.uniform(1, 2) * 2.0 ** e)
            step = max(np.spacing(np.abs(top)), np.float32(1.0))
            rows.append(np.float32(np.round(top / step) * step) - step * g.integers(0, 3, E).astype(np.float32))
    return torch.from_numpy(np.stack(rows).astype(np.float32))


def test_forward_logits_of_any_size(gpu):
    l = far_rows(1)
    ids = torch.randint(0, 24, (len(l), 3), generator=torch.Generator().manual_seed(1))
    for score in ("softmax", "sigmoid"):
        check_forward(l, ids, torch.arange(len(l) + 1), gpu, score, len(l))


@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_gradient_logits_of_any_size(gpu, score, renorm):
    l = far_rows(2)
    g = torch.Generator().manual_seed(2)
    ids = torch.stack([torch.randperm(24, generator=g)[:3] for _ in range(len(l))])
    check_gradient(l, ids, None, gpu, score, renorm, 1.0, 1, ("loss", "w"))
    if score == "softmax":
        keep = l.abs().amax(1) < 2.0 ** 63  # d_z and the logarithm stay finite
        check_gradient(l[keep], ids[keep], None, gpu, score, renorm, 1.0, 1, ("z",))


def test_z_of_rows_without_a_logarithm(gpu):
    """A NaN makes z NaN, whatever stands beside it, and +infinity makes it infinite."""
    l = torch.zeros(6, 16)
    l[0, 3], l[1], l[1, 5], l[2], l[2, 6], l[3], l[3, 0] = NAN, -INF, NAN, 2.0 ** 110, NAN, -(2.0 ** 40), NAN
    l[4, 2] = INF
    ids = torch.zeros(6, 2, dtype=torch.int64)
    out = forward(*on(gpu, l, ids, torch.arange(7)), gpu, S=6)
    z = out["z"].cpu()
    assert torch.isnan(z[:4]).all() and torch.isinf(z[4]) and abs(z[5].item() - np.log(16) ** 2) < 1e-5
    assert torch.isnan(out["share"][:5]).all()


# ---- sigmoid scores far below the row's largest

def low_rows(E=24):
    """Whole numbers, so that distances are exact: tops from 2 to -200 and scores down to exp(-60) of them."""
    g = np.random.default_rng(3)
    tops = [2, 0, -1, -5, -20, -30, -40, -50, -59, -60, -61, -90, -150, -200]
    l = np.stack([t - g.integers(0, 61, E) for t in tops]).astype(np.float32)
    l[:, 0], l[:, 1] = tops, np.array(tops) - 60
    return torch.from_numpy(l)


def test_forward_low_sigmoid_scores(gpu):
    l = low_rows()
    check_forward(l, torch.zeros(len(l), 2, dtype=torch.int64), torch.arange(len(l) + 1), gpu, "sigmoid", len(l))


@pytest.mark.parametrize("ids", [[0, 1, 2], [1, 2, 3], [1, 5, 6]])
def test_gradient_low_sigmoid_scores(gpu, ids):
    l = low_rows()
    check_gradient(l, torch.tensor([ids] * len(l)), None, gpu, "sigmoid", True, 1.0, 1, ("loss", "w"))
    check_gradient(l, torch.tensor([ids] * len(l)), None, gpu, "sigmoid", True, 1.0, 1, ("w",))


# ---- entries that take no part

@pytest.mark.parametrize("E", [24, 33, 300])
@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_gradient_of_entries_without_a_weight(gpu, score, renorm, value, E):
    """What stands at ids that are none, or whose logit is masked, is not read into the row."""
    l, ids, _ = inputs(40, E, 5, 5)
    ids[3, 1], ids[4, 0], ids[5, 2], ids[6] = -1, E, 1 << 40, -1
    l[7, ids[7, 2]] = -INF
    l[8, ids[8]] = -INF
    l[9] = -INF
    l[10] -= 300.0  # sums of the chosen that are formed again
    ids[10, 4] = -1
    l[11, ids[11, 1:]] = -INF
    d = torch.randn(40, 5, generator=torch.Generator().manual_seed(6))
    none = (ids < 0) | (ids >= E) | (l.gather(1, ids.clamp(0, E - 1)) == -INF)
    assert none.sum() > 20
    want = gradient(*on(gpu, l, ids, None), gpu, score=score, renormalize=renorm, d_topk_w=d.masked_fill(none, 0.0).to(gpu))
    got = gradient(*on(gpu, l, ids, None), gpu, score=score, renormalize=renorm, d_topk_w=d.masked_fill(none, value).to(gpu))
    assert torch.isfinite(want).all() and torch.equal(got, want)


@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_gradient_of_rows_with_a_nan_and_unused_entries(gpu, score, renorm):
    """Neither reaches another row, wherever it lies in the workgroup."""
    for E in (8, 33, 64, 200):
        l, ids, _ = inputs(50, E, 4, 7)
        ids[::3, 1], ids[::3, 3] = -1, E
        d = torch.randn(50, 4, generator=torch.Generator().manual_seed(8)).to(gpu)
        want = gradient(*on(gpu, l, ids, None), gpu, score=score, renormalize=renorm, d_topk_w=d)
        l[::3, 2] = NAN
        got = gradient(*on(gpu, l, ids, None), gpu, score=score, renormalize=renorm, d_topk_w=d)
        bad = torch.arange(50, device=gpu) % 3 == 0
        assert torch.equal(got[~bad], want[~bad]) and torch.isfinite(want).all() and torch.isnan(got[bad]).any(1).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(20, 3), (33, 8), (64, 20), (257, 6), (1000, 9)])
def test_gradient_of_rows_one_after_another(gpu, E, k, score, renorm):
    """Rows that a group of lanes takes in turn, through the same LDS, have the bits that they have alone; ids twice, and
    the same ones in rows that follow each other."""
    T = 70001 if E <= 64 else 20011
    g = torch.Generator(gpu).manual_seed(E)
    l = torch.randn(T, E, generator=g, device=gpu)
    ids = torch.randint(-1, E, (T, k), generator=g, device=gpu)
    ids[T // 2:] = ids[0]
    l[::3] = l[::3].scatter(1, ids[::3].clamp_min(0), -130.0)  # weights that are formed again
    d = torch.randn(T, k, generator=g, device=gpu)
    whole = gradient(l, ids, None, gpu, score=score, renormalize=renorm, d_topk_w=d)
    for at in range(0, T, 4000):
        part = slice(at, min(at + 4000, T))
        alone = gradient(l[part], ids[part], None, gpu, score=score, renormalize=renorm, d_topk_w=d[part])
        assert torch.equal(whole[part], alone), at
