"""Argument checks of the microscaled and balance calls: the C ABI's statuses and the binding's errors (no GPU)."""
import ctypes

import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)       # 8-byte aligned only
BAD = ctypes.c_void_p(0x10001)


def quant(shape, x=FAKE, q=FAKE, sf=FAKE, dq=None):
    return B.lib().moe_mx_quant(ctypes.byref(shape), x, q, sf, dq, None)


QUANT = dict(num_rows=4, num_cols=256)


@pytest.mark.parametrize("change,status", [
    (dict(num_rows=-1), -2), (dict(num_rows=1 << 28), -2), (dict(num_cols=0), -2), (dict(num_cols=-32), -2),
    (dict(num_cols=(1 << 20) + 32), -2), (dict(num_cols=48), -3), (dict(x_stride=255), -2), (dict(x_stride=-256), -2),
    (dict(x_stride=260), -3), (dict(x_stride=1 << 41), -2)])
def test_quant_shapes(change, status):
    assert quant(B.make_mx_quant(**{**QUANT, **change})) == status


@pytest.mark.parametrize("field", ["x_type", "format"])
def test_quant_types(field):
    for bad in (-1, 2):
        s = B.make_mx_quant(**QUANT)
        setattr(s, field, bad)
        assert quant(s) == -2


def test_quant_pointers():
    s = B.make_mx_quant(**QUANT)
    assert B.lib().moe_mx_quant(None, FAKE, FAKE, FAKE, None, None) == -1
    assert quant(s, x=None) == -1 and quant(s, q=None) == -1 and quant(s, sf=None) == -1
    assert quant(s, q=None, sf=None) == -1                       # nothing to write
    for name in ("x", "q", "dq"):
        assert quant(s, **{name: ODD}) == -3, name
    assert quant(B.make_mx_quant(0, 256), None, None, None) == 0


def linear(shape, x=FAKE, sf=FAKE, w=FAKE, y=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return B.lib().moe_mx_linear(ctypes.byref(shape), x, sf, w, y, ws, ws_bytes, None)


LINEAR = dict(num_tokens=4, in_features=256, out_features=48)


@pytest.mark.parametrize("change,status", [
    (dict(num_tokens=-1), -2), (dict(num_tokens=1 << 28), -2), (dict(in_features=0), -2), (dict(in_features=40), -3),
    (dict(in_features=(1 << 20) + 32), -2), (dict(out_features=0), -2), (dict(out_features=(1 << 20) + 1), -2),
    (dict(y_stride=47), -2), (dict(y_stride=-48), -2), (dict(y_stride=1 << 41), -2)])
def test_linear_shapes(change, status):
    s = B.make_mx_linear(**{**LINEAR, **change})
    v, i = ctypes.c_size_t(), ctypes.c_int32()
    lib = B.lib()
    assert linear(s) == status
    for f in (lib.moe_mx_linear_weight_bytes, lib.moe_mx_linear_workspace_bytes, lib.moe_mx_linear_max_workspace_bytes):
        assert f(ctypes.byref(s), ctypes.byref(v)) == status
    assert lib.moe_mx_linear_tile(ctypes.byref(s), *[ctypes.byref(i)] * 3) == status
    assert lib.moe_mx_linear_prepare(ctypes.byref(s), FAKE, FAKE, FAKE, None) == status


def test_linear_pointers():
    s, lib = B.make_mx_linear(**LINEAR), B.lib()
    assert lib.moe_mx_linear(None, FAKE, FAKE, FAKE, FAKE, FAKE, 0, None) == -1
    for f in (lib.moe_mx_linear_weight_bytes, lib.moe_mx_linear_workspace_bytes, lib.moe_mx_linear_max_workspace_bytes):
        assert f(ctypes.byref(s), None) == -1
    i = ctypes.c_int32()
    assert lib.moe_mx_linear_tile(ctypes.byref(s), None, ctypes.byref(i), ctypes.byref(i)) == -1
    for at in range(3):
        a = [FAKE] * 3
        a[at] = None
        assert lib.moe_mx_linear_prepare(ctypes.byref(s), *a, None) == -1
    assert lib.moe_mx_linear_prepare(ctypes.byref(s), ODD, FAKE, FAKE, None) == -3
    assert lib.moe_mx_linear_prepare(ctypes.byref(s), FAKE, FAKE, ODD, None) == -3
    for name in ("x", "sf", "w", "y"):
        assert linear(s, **{name: None}) == -1 and linear(s, **{name: BAD}) == -3, name
    assert linear(s, x=ODD) == -3 and linear(s, w=ODD) == -3
    s.x_format = 2
    assert linear(s) == -2
    assert linear(B.make_mx_linear(0, 256, 48), None, None, None, None, None, 0) == 0


def test_linear_weight_bytes():
    assert B.mx_linear_weight_bytes(B.make_mx_linear(1, 128, 64)) == 64 * (64 + 4)
    assert B.mx_linear_weight_bytes(B.make_mx_linear(1, 160, 65)) == 128 * 2 * (64 + 4)


def test_linear_workspaces():
    """A workspace that is missing, misaligned or a byte short is refused; the largest serves every smaller batch."""
    seen = 0
    for fmt in ("e2m1", "e4m3"):
        for K, N in ((32, 1), (96, 70), (7168, 64), (7168, 4096), (4064, 1537), (2048, 7168), (1 << 20, 64), (64, 1 << 20)):
            most = B.mx_linear_max_workspace_bytes(B.make_mx_linear(20000, K, N, fmt))
            for T in list(range(0, 70)) + [127, 128, 129, 255, 256, 257, 511, 1000, 1024, 1025, 2047, 4097, 9999, 16384, 20000]:
                s = B.make_mx_linear(T, K, N, fmt)
                need = B.mx_linear_workspace_bytes(s)
                assert need <= most, (fmt, T, K, N)
                if need and T:
                    seen += 1
                    assert linear(s, ws=None) == -1 and linear(s, ws=ODD) == -3 and linear(s, ws_bytes=need - 1) == -4
    assert seen
    for K, N in ((1 << 20, 1 << 20), (32, 1), (7168, 1 << 20), (96, 1)):  # the sizes at the limits are formed at all
        assert B.mx_linear_max_workspace_bytes(B.make_mx_linear((1 << 28) - 1, K, N)) >= \
            B.mx_linear_workspace_bytes(B.make_mx_linear((1 << 28) - 1, K, N))


def balance(shape, logits=FAKE, ids=FAKE, off=None, counts=FAKE, rows=FAKE, share=FAKE, loss=FAKE, z=None, ws=FAKE,
            ws_bytes=1 << 40):
    return B.lib().moe_balance(ctypes.byref(shape), logits, ids, off, counts, rows, share, loss, z, ws, ws_bytes, None)


def grad(shape, logits=FAKE, ids=FAKE, off=None, counts=FAKE, rows=FAKE, d_loss=FAKE, d_z=None, d_w=FAKE, out=FAKE):
    return B.lib().moe_gate_grad(ctypes.byref(shape), logits, ids, off, counts, rows, d_loss, d_z, d_w, out, None)


BALANCE = dict(num_tokens=4, num_experts=32, topk=4)


@pytest.mark.parametrize("change,status", [
    (dict(num_tokens=-1), -2), (dict(num_tokens=1 << 28), -2), (dict(num_tokens=(1 << 28) - 1, topk=5), -2), (dict(num_experts=0), -2),
    (dict(num_experts=1025), -2), (dict(topk=0), -2), (dict(topk=33), -2), (dict(num_experts=1024, topk=65), -2),
    (dict(num_seqs=0), -2), (dict(num_seqs=(1 << 20) + 1), -2), (dict(num_seqs=1 << 20, num_experts=1024), -2),
    (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2), (dict(logits_stride=31), -2),
    (dict(logits_stride=1 << 41), -2)])
def test_balance_shapes(change, status):
    s = B.make_balance(**{**BALANCE, **change})
    assert balance(s, off=FAKE) == status and grad(s, off=FAKE) == status
    v = ctypes.c_size_t()
    assert B.lib().moe_balance_workspace_bytes(ctypes.byref(s), ctypes.byref(v)) == status


@pytest.mark.parametrize("field", ["score", "renormalize", "logits_type"])
def test_balance_types(field):
    for bad in (-1, 2):
        s = B.make_balance(**BALANCE)
        setattr(s, field, bad)
        assert balance(s) == -2 and grad(s) == -2


def test_balance_pointers():
    s, lib = B.make_balance(**BALANCE), B.lib()
    assert lib.moe_balance(None, *[FAKE] * 9, 0, None) == -1 and lib.moe_gate_grad(None, *[FAKE] * 9, None) == -1
    assert lib.moe_balance_workspace_bytes(ctypes.byref(s), None) == -1
    for name in ("logits", "ids", "ws"):
        assert balance(s, **{name: None}) == -1, name
    assert balance(s, counts=None, rows=None, share=None, loss=None) == -1
    for name in ("logits", "ids", "off", "counts", "rows", "share", "loss", "z", "ws"):
        assert balance(s, **{name: BAD}) == -3, name
    assert balance(s, ws=ODD) == -3
    assert balance(s, ws_bytes=B.balance_workspace_bytes(s) - 1) == -4
    assert balance(B.make_balance(**BALANCE, num_seqs=2)) == -2           # two sequences without offsets
    assert balance(B.make_balance(**BALANCE, score="sigmoid"), z=FAKE) == -2

    for name in ("logits", "ids", "counts", "rows", "out"):
        assert grad(s, **{name: None}) == -1, name
    assert grad(s, d_loss=None, d_w=None) == -1
    assert grad(s, d_loss=None, d_z=FAKE, counts=None, rows=None) == -1
    for name in ("logits", "ids", "off", "counts", "rows", "d_loss", "d_z", "d_w", "out"):
        assert grad(s, **{name: BAD}) == -3, name
    assert grad(B.make_balance(**BALANCE, num_seqs=2)) == -2
    assert grad(B.make_balance(**BALANCE, score="sigmoid"), d_z=FAKE) == -2
    assert grad(B.make_balance(**BALANCE, logits_stride=40), out=FAKE) == -2  # in place of rows that lie apart
    assert grad(B.make_balance(0, 32, 4), None, None, None, None, None, FAKE, None, None, None) == 0


@pytest.mark.parametrize("T,E,S", [(0, 1, 1), (1, 1024, 1), (65536, 384, 1), ((1 << 24), 64, 1000), ((1 << 28) - 1, 1, 1),
                                   (5, 1023, 1 << 20)])
def test_balance_workspace(T, E, S):
    """Less than the logits themselves take, beside what every sequence has."""
    b = B.balance_workspace_bytes(B.make_balance(T, E, 1, num_seqs=S))
    assert 0 < b < 4096 + S * (16 * E + 64) + 8192 * (E + 1) + (T // 128) * (E + 1)


class Cpu:
    """What the binding checks before it reaches the library: tensors that are not on the device."""
    t = torch.zeros(4, 256, dtype=torch.bfloat16)


def test_binding_refuses_host_tensors():
    u8 = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.mx_quant(B.make_mx_quant(4, 256), Cpu.t, u8, u8)
    with pytest.raises(ValueError):
        B.mx_linear_prepare(B.make_mx_linear(4, 256, 4), u8, u8)
    with pytest.raises(ValueError):
        B.mx_linear(B.make_mx_linear(4, 256, 4), u8, u8, u8, Cpu.t)
    with pytest.raises(ValueError):
        B.balance(B.make_balance(4, 8, 2), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64), u8)
    with pytest.raises(ValueError):
        B.gate_grad(B.make_balance(4, 8, 2), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        B.mx_quant(B.make_mx_quant(4, 256), None, u8, u8)
    with pytest.raises(KeyError):
        B.make_mx_quant(4, 256, format="e5m2")
    with pytest.raises(KeyError):
        B.make_balance(4, 8, 2, score="tanh")
