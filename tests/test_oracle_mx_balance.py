"""Pins of the oracle of microscaled quantisation, the balance of the load and the gate's gradient (no GPU)."""
import itertools

import numpy as np
import pytest
import torch

from oracle.balance import balance_ref, gate_grad_ref, objective
from oracle.formats import E2M1_TABLE
from oracle.front import gate_ref
from oracle.mx import encode_e2m1_rne, mx_quant_ref


def test_e2m1_codes_and_ties():
    assert np.array_equal(encode_e2m1_rne(E2M1_TABLE), np.arange(16))
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for v, c in ties.items():
        assert encode_e2m1_rne(np.array([v, -v])).tolist() == [c, c | 8]
        assert encode_e2m1_rne(np.nextafter(v, 0)) == (c if c * 2 == 0 or E2M1_TABLE[c] < v else c - 1)
        assert encode_e2m1_rne(np.nextafter(v, 9)) == (c if E2M1_TABLE[c] > v else c + 1)


@pytest.mark.parametrize("fmt,most", [("e2m1", 6.0), ("e4m3", 448.0)])
def test_scales(fmt, most):
    for e in (-130, -127, -100, 0, 5, 100):
        x = np.zeros((3, 32))
        x[0, 3], x[1, 3], x[2, 3] = most * 2.0 ** e, np.nextafter(most * 2.0 ** e, np.inf), -most * 2.0 ** e
        assert mx_quant_ref(x, fmt)[1][:, 0].tolist() == [max(e, -127) + 127, max(e + 1, -127) + 127, max(e, -127) + 127]
    assert mx_quant_ref(np.zeros((1, 32)), fmt)[1].tolist() == [[0]]
    x = np.ones((2, 64))
    x[0, 5], x[1, 40] = np.nan, np.inf
    c, s, d = mx_quant_ref(x, fmt)
    assert s[0, 0] == 255 and s[1, 1] == 255 and s[0, 1] != 255
    assert np.isnan(d[0, :32]).all() and np.isnan(d[1, 32:]).all() and (d[0, 32:] == 1).all() and not c[0, :32].any()


def test_e4m3_against_torch():
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    c, s, _ = mx_quant_ref(x.numpy(), "e4m3")
    v = np.ldexp(x.numpy().reshape(64, 8, 32), -(s.astype(int) - 127)[..., None]).reshape(64, 256)
    assert np.array_equal(torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), c)


def case(seed, T, E, k, hole, S):
    g = np.random.default_rng(seed)
    l = g.normal(size=(T, E))
    if hole:
        l[g.random((T, E)) < hole] = -np.inf
        l[T // 2] = -np.inf
    ids = gate_ref(l, k)[0]
    off = None if S == 1 else np.sort(g.integers(0, T + 1, S + 1))
    return l, ids, off, g


@pytest.mark.parametrize("score,hole,S", itertools.product(["softmax", "sigmoid"], [0.0, 0.2], [1, 4]))
def test_balance_against_torch(score, hole, S):
    l, ids, off, _ = case(1, 40, 12, 3, hole, S)
    r = balance_ref(l, ids, off, score)
    o = [0, 40] if off is None else off.tolist()
    for s, (a, b) in enumerate(zip(o, o[1:])):
        x = torch.from_numpy(l[a:b])
        x = x[(x > -np.inf).any(1)]
        p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x) / torch.sigmoid(x).sum(1, keepdim=True)
        c = torch.bincount(torch.from_numpy(ids[a:b])[torch.from_numpy(ids[a:b]) >= 0].flatten(), minlength=12)
        assert r["counts"][s].tolist() == c.tolist() and r["rows"][s] == len(x)
        if len(x):
            assert np.allclose(r["share"][s], p.mean(0).numpy(), rtol=1e-12, atol=0)
            assert np.isclose(r["loss"][s], 12 * float((c.double() / c.sum()) @ p.mean(0)), rtol=1e-12)
            if score == "softmax":
                assert np.isclose(r["z"][s], float(torch.logsumexp(x, 1).square().mean()), rtol=1e-12)


@pytest.mark.parametrize("score,renorm,hole", itertools.product(["softmax", "sigmoid"], [True, False], [0.0, 0.2]))
def test_gradient_against_differences(score, renorm, hole):
    """Central differences of the objective, whose error is h^2 / 6 of a third derivative of order 1, and 2^-52 / h."""
    l, ids, off, g = case(2, 9, 6, 3, hole, 3)
    ids[1, 1] = ids[1, 0]  # an id twice, and one that is none
    ids[2, 0] = 6
    b = balance_ref(l, ids, off, score)
    kw = dict(d_loss=g.normal(size=3), d_topk_w=g.normal(size=(9, 3)), offsets=off, score=score, renormalize=renorm, scale=1.5)
    if score == "softmax":
        kw["d_z"] = g.normal(size=3)
    grad = gate_grad_ref(l, ids, b["counts"], b["rows"], **kw)
    h = 1e-5
    for t in range(9):
        for e in range(6):
            if np.isneginf(l[t, e]) or np.isnan(grad[t, e]):
                assert grad[t, e] == 0 or np.isnan(grad[t, e])
                continue
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = (objective(up, ids, b["counts"], b["rows"], **kw) - objective(dn, ids, b["counts"], b["rows"], **kw)) / (2 * h)
            assert abs(d - grad[t, e]) < 1e-8, (t, e)


def test_even_load_has_loss_one_and_no_gradient():
    l = np.random.default_rng(3).normal(size=(8, 4))
    counts = np.full((1, 4), 2)
    assert np.abs(gate_grad_ref(l, np.zeros((8, 1), int), counts, [8], d_loss=[1.0])).max() < 1e-16
    l[:] = 0.0
    assert balance_ref(l, np.arange(8)[:, None] % 4)["loss"] == [1.0]
