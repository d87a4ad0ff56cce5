"""Pins of the oracle's norm, router product and gate (CPU)."""
import itertools

import numpy as np
import pytest
import torch

from oracle.front import gate_ref, norm_ref, router_ref, scores_ref


def test_norm_against_torch():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 96, generator=g, dtype=torch.float64) * 3
    r = torch.randn(9, 96, generator=g, dtype=torch.float64)
    w = torch.randn(96, generator=g, dtype=torch.float64)
    h, v, code, scaled = norm_ref(x.numpy(), w.numpy(), 1e-5, r.numpy())
    want = torch.nn.functional.rms_norm(x + r, (96,), w, 1e-5)
    np.testing.assert_allclose(v, want.numpy(), rtol=1e-13)
    np.testing.assert_array_equal(h, (x + r).numpy())
    top = np.abs(scaled).reshape(9, 3, 32).max(axis=2)
    assert (top <= 448).all() and (top > 224).all()        # the next smaller power of two would not fit
    np.testing.assert_allclose(scaled * np.repeat(2.0 ** (code.astype(float) - 127), 32, axis=1), v, rtol=1e-15)


def test_norm_scale_border_and_zero_blocks():
    x = np.zeros((1, 96))
    x[0, 0], x[0, 32] = 448.0, np.nextafter(448.0, 500)
    w = np.ones(96)
    rms = np.sqrt((x ** 2).mean())
    _, v, code, _ = norm_ref(x, w * rms, 0.0)              # v = x
    np.testing.assert_allclose(v, x, rtol=1e-15)
    assert code[0, 2] == 0                                 # a block of zeros
    _, _, code, _ = norm_ref(np.full((1, 32), 7.0), np.full(32, 448.0), 0.0)
    assert code[0, 0] == 127                               # v = 448 exactly: scale 1
    _, _, code, _ = norm_ref(np.full((1, 32), 7.0), np.full(32, np.nextafter(448.0, 500)), 0.0)
    assert code[0, 0] == 128


def test_router_and_scores_against_torch():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(5, 64, generator=g, dtype=torch.float64), torch.randn(7, 64, generator=g, dtype=torch.float64)
    np.testing.assert_allclose(router_ref(x.numpy(), w.numpy()), torch.nn.functional.linear(x, w).numpy(), rtol=1e-12)
    l = torch.randn(6, 9, generator=g, dtype=torch.float64) * 4
    np.testing.assert_allclose(scores_ref(l.numpy(), "softmax"), torch.softmax(l, -1).numpy(), rtol=1e-14)
    np.testing.assert_allclose(scores_ref(l.numpy(), "sigmoid"), torch.sigmoid(l).numpy(), rtol=1e-14)


def test_gate_against_topk():
    l = torch.randn(50, 12, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    p = torch.softmax(l, -1)
    v, i = torch.topk(p, 4)
    ids, w = gate_ref(l.numpy(), 4, renormalize=False, scale=2.5)
    np.testing.assert_array_equal(ids, i.numpy())
    np.testing.assert_allclose(w, 2.5 * v.numpy(), rtol=1e-13)
    ids, w = gate_ref(l.numpy(), 4)
    np.testing.assert_allclose(w, (v / v.sum(-1, keepdim=True)).numpy(), rtol=1e-13)


@pytest.mark.parametrize("group_score,kept,biased", list(itertools.product(["max", "top2"], [1, 2], [False, True])))
def test_gate_groups_by_brute_force(group_score, kept, biased):
    """Over every choice of groups: the kept set has the largest marks, and the ids are its largest c."""
    rng = np.random.default_rng(4)
    E, G, k = 12, 4, 3
    for _ in range(40):
        l = rng.standard_normal(E)
        b = rng.integers(-3, 4, E) * 0.1 if biased else None
        s = 1 / (1 + np.exp(-l))
        c = s + b if biased else l
        m = s if group_score == "top2" and not biased else c
        per = np.sort(m.reshape(G, 3), axis=1)[:, ::-1]
        mark = per[:, 0] + (per[:, 1] if group_score == "top2" else 0)
        best = max(itertools.combinations(range(G), kept), key=lambda q: sum(mark[list(q)]))
        cand = [e for e in range(E) if e // 3 in best]
        want = sorted(cand, key=lambda e: -c[e])[:k]
        ids, _ = gate_ref(l[None], k, "sigmoid", b, G, kept, group_score)
        assert list(ids[0]) == want


def test_gate_ties_masks_and_nan():
    inf, nan = np.inf, np.nan
    l = np.array([[1.0, 2.0, 2.0, 1.0], [-inf, 0.5, -inf, -inf], [-inf] * 4, [0.0, -0.0, 0.0, -0.0], [1.0, nan, 3.0, 2.0]])
    ids, w = gate_ref(l, 3, "sigmoid")
    np.testing.assert_array_equal(ids, [[1, 2, 0], [1, -1, -1], [-1, -1, -1], [0, 1, 2], [1, 2, 3]])
    np.testing.assert_array_equal(w[1:3], [[1, 0, 0], [0, 0, 0]])
    assert np.isnan(w[4]).all()
    ids, w = gate_ref(l, 3, "sigmoid", renormalize=False)
    assert np.isnan(w[4, 0]) and np.isfinite(w[4, 1:]).all()
    # a bias of -inf masks an expert; a group of masked experts is never kept
    ids, _ = gate_ref(np.array([[5.0, 4.0, 1.0, 2.0]]), 2, "softmax", np.array([-inf, -inf, 0, 0]), 2, 1)
    np.testing.assert_array_equal(ids, [[3, 2]])
