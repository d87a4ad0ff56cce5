"""GPU parity of moe_mx_quant and moe_mx_linear with the float64 oracle.

Quantisation is one rounding of an exact quotient: codes, scales and values are equal.  The product: BF16's rounding,
half a step of 2^-8 of the value, and the sum's: one FP32 rounding for each of the 2 KT instructions of a tile and of the
partial sums, 2^-24 of the sum of magnitudes each, and inside an instruction with E4M3 activations 2^-13 of it.
"""
import itertools

import numpy as np
import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B
from oracle.formats import E2M1_TABLE, E4M3_TABLE, unpack_fp4
from oracle.mx import mx_quant_ref

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def quantised(x, fmt, dq=True, codes=True, stride=0):
    R, C = x.shape
    s = B.make_mx_quant(R, C, fmt, x.dtype, stride)
    q = torch.full((R, C // 2 if fmt == "e2m1" else C), 0xEE, dtype=torch.uint8, device=x.device) if codes else None
    sf = torch.full((R, C // 32), 0xEE, dtype=torch.uint8, device=x.device) if codes else None
    d = torch.full((R, C), 7.0, dtype=BF16, device=x.device) if dq else None
    B.mx_quant(s, x, q, sf, d)
    return q, sf, d


def check_quant(x, fmt, stride=0):
    q, sf, d = quantised(x, fmt, stride=stride)
    rq, rsf, rd = mx_quant_ref(x.double().cpu().numpy(), fmt)
    got = unpack_fp4(q.cpu().numpy()) if fmt == "e2m1" else q.cpu().numpy()
    assert np.array_equal(sf.cpu().numpy(), rsf)
    assert np.array_equal(got, rq)
    assert np.array_equal(d.float().cpu().numpy(), rd, equal_nan=True)
    return q, sf, d


SHAPES = [(1, 32), (3, 64), (1, 96), (2, 2048), (5, 2080), (130, 160), (7, 4064), (33, 7168), (1000, 32), (2, 1 << 20)]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,C", SHAPES)
def test_quant_sizes(gpu, R, C, dtype, fmt):
    print(f"quant {R} x {C} {dtype} {fmt}", flush=True)
    x = torch.randn(R, C, generator=gen(R + C)) * torch.exp2(torch.randint(-40, 40, (R, C // 32, 1), generator=gen(C)).float()
                                                             ).expand(R, C // 32, 32).reshape(R, C)
    check_quant(x.to(dtype).to(gpu), fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("R,C,stride", [(4, 64, 72), (9, 2080, 4160), (1, 32, 40), (70, 128, 136)])
def test_quant_strided_rows(gpu, R, C, stride, fmt):
    x = torch.randn(R, stride, generator=gen(R)).to(BF16).to(gpu)
    x[:, C:] = float("nan")  # never read into a block
    check_quant(x[:, :C], fmt, stride=stride)


@pytest.mark.parametrize("fmt,most", [("e2m1", 6.0), ("e4m3", 448.0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_every_border(gpu, dtype, fmt, most):
    """Ties and their neighbours at every step of the format, maxima at, under and over a power's border, both signs,
    over all scales, subnormals and the largest numbers among them."""
    table = E2M1_TABLE[:8] if fmt == "e2m1" else E4M3_TABLE[:127]
    mids = torch.from_numpy((table[1:] + table[:-1]) / 2).to(F32)
    v = torch.cat([mids, torch.from_numpy(table).to(F32)])
    if dtype == F32:
        v = torch.cat([v, torch.nextafter(v, torch.tensor(9e9)), torch.nextafter(v, torch.tensor(-9e9))])
    v = v[v.abs() <= most]
    v = torch.cat([v, -v])
    v = torch.cat([v, torch.zeros(-len(v) % 31)]).view(-1, 31)
    rows = []
    for e in (-149, -140, -133, -127, -126, -100, -1, 0, 1, 60, 118, 119, 120, 125):
        for top in (most, most / 2 * (1 + 2.0 ** -7), most / 2):
            rows.append(torch.cat([torch.full((len(v), 1), top), v * (1.0 if top == most else 0.5)], 1).double() * 2.0 ** e)
    x = torch.cat(rows)
    x = x[(x.abs() <= torch.finfo(dtype).max).all(1)].to(dtype)
    x = torch.cat([x, torch.full((1, 32), torch.finfo(dtype).max, dtype=dtype), torch.full((1, 32), torch.finfo(dtype).smallest_normal * 2 ** -7, dtype=dtype)])
    check_quant(x.to(gpu), fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_without_finite_values(gpu, dtype, fmt):
    x = torch.randn(6, 96, generator=gen(4)).to(dtype)
    x[0, 40], x[1, 0], x[2, 95], x[3] = float("nan"), float("inf"), -float("inf"), 0.0
    x[4, 32:64] = -0.0
    x[5] = float("nan")
    check_quant(x.to(gpu), fmt)


def test_quant_outputs_apart(gpu):
    x = torch.randn(17, 160, generator=gen(5)).to(BF16).to(gpu)
    for fmt in ("e2m1", "e4m3"):
        q, sf, d = quantised(x, fmt)
        q1, sf1, _ = quantised(x, fmt, dq=False)
        _, _, d1 = quantised(x, fmt, codes=False)
        assert torch.equal(q, q1) and torch.equal(sf, sf1) and torch.equal(d, d1)


# ---- product

def values(q, sf, fmt):
    table = torch.from_numpy(E2M1_TABLE if fmt == "e2m1" else E4M3_TABLE).to(q.device)
    v = table[(torch.stack([q & 15, q >> 4], -1).flatten(1) if fmt == "e2m1" else q).long()]
    s = torch.exp2(sf.double() - 127)
    s[sf == 255] = float("nan")
    return v * s.repeat_interleave(32, 1)


def operands(T, K, N, fmt, seed, gpu, spread=2):
    """Codes of normal values with an uneven scale per block."""
    g = gen(seed)
    x = torch.randn(T, K, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (T, K // 32, 1), generator=g).float()
                                                    ).expand(T, K // 32, 32).reshape(T, K)
    w = torch.randn(N, K, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (N, K // 32, 1), generator=g).float()
                                                    ).expand(N, K // 32, 32).reshape(N, K)
    return quantised(x.to(gpu), fmt, dq=False)[:2], quantised(w.to(gpu), "e2m1", dq=False)[:2]


def product(x, w, fmt, y_stride=0, ws_fill=0xFF):
    (q, sf), (wq, wsf) = x, w
    T, K, N = q.shape[0], sf.shape[1] * 32, wq.shape[0]
    s = B.make_mx_linear(T, K, N, fmt, y_stride)
    y = torch.full((T, y_stride or N), 7.0, dtype=BF16, device=q.device)
    ws = torch.full((B.mx_linear_workspace_bytes(s),), ws_fill, dtype=torch.uint8, device=q.device)
    B.mx_linear(s, q, sf, B.mx_linear_prepare(s, wq, wsf), y[:, :N], ws)
    if y_stride:
        assert (y[:, N:] == 7).all()  # what lies between the rows stays
    return y[:, :N], s


def check_product(T, K, N, fmt, gpu, seed=0, y_stride=0, spread=2):
    x, w = operands(T, K, N, fmt, seed + T + K + N, gpu, spread)
    y, s = product(x, w, fmt, y_stride)
    xv, wv = values(*x, fmt), values(*w, "e2m1")
    ref, mag = xv @ wv.t().contiguous(), xv.abs() @ wv.abs().t().contiguous()
    steps = 2 * ((K + 127) // 128) + B.mx_linear_tile(s)[2]
    tol = 2.0 ** -8 * ref.abs() + (steps * 2.0 ** -24 + (2.0 ** -13 if fmt == "e4m3" else 0.0)) * 1.01 * mag
    off = (y.double() - ref).abs()
    assert (off <= tol).all(), f"{((off - tol) / mag).max():.2e} of the magnitudes over, at {int((off - tol).argmax())}"
    return y


LINEARS = [(1, 32, 1), (1, 7168, 96), (2, 64, 33), (3, 96, 2), (15, 512, 100), (16, 1024, 64), (17, 160, 63), (31, 4064, 257), (32, 2048, 130),
           (33, 288, 65), (48, 640, 200), (64, 4096, 192), (65, 128, 64), (100, 7168, 70), (128, 2048, 512), (129, 256, 130), (255, 32, 129),
           (300, 4064, 257), (513, 544, 257), (1000, 96, 1000), (2047, 128, 1537)]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,K,N", LINEARS)
def test_linear_sizes(gpu, T, K, N, fmt):
    print(f"linear {T} x {K} x {N} {fmt}", flush=True)
    check_product(T, K, N, fmt, gpu)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,K,N", [(4097, 160, 4000), (8192, 512, 2048), (2049, 1056, 8192), (16384, 64, 1030)])
def test_linear_many_tiles(gpu, T, K, N, fmt):
    print(f"linear {T} x {K} x {N} {fmt}", flush=True)
    check_product(T, K, N, fmt, gpu)


@pytest.mark.parametrize("T", list(range(1, 40)) + [47, 63, 64, 66, 80, 96, 97, 112, 127, 160, 192, 256])
def test_linear_every_small_batch(gpu, T):
    print(f"linear {T}", flush=True)
    for fmt in ("e2m1", "e4m3"):
        check_product(T, 1184, 136, fmt, gpu)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,K,N,stride", [(5, 256, 31, 33), (40, 256, 64, 70), (130, 96, 100, 101), (300, 128, 63, 64), (4097, 64, 4001, 4003)])
def test_linear_strided_output(gpu, T, K, N, stride, fmt):
    check_product(T, K, N, fmt, gpu, y_stride=stride)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_linear_far_scales(gpu, fmt):
    check_product(70, 1024, 130, fmt, gpu, spread=14)


@pytest.mark.parametrize("T", [1, 20, 130, 4100])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_linear_nan(gpu, T, fmt):
    """A NaN scale or code reaches its row, or its output, and no other; the last K-step is a part of one."""
    K, N = 160, 4100 if T > 4000 else 70
    x, w = operands(T, K, N, fmt, 3, gpu)
    clean, _ = product(x, w, fmt)
    (q, sf), (wq, wsf) = x, w
    sf[T // 2, 4] = 255
    if fmt == "e4m3" and T > 1:
        q[T - 1, K - 1] = 0x7F
    y, _ = product(x, w, fmt)
    bad = torch.zeros(T, dtype=torch.bool, device=gpu)
    bad[T // 2] = True
    if fmt == "e4m3" and T > 1:
        bad[T - 1] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])
    x, w = operands(T, K, N, fmt, 3, gpu)
    w[1][N - 1, 0] = 255
    y, _ = product(x, w, fmt)
    assert torch.isnan(y[:, N - 1]).all() and torch.equal(y[:, :N - 1], clean[:, :N - 1])


def test_linear_workspace_is_not_read(gpu):
    used = 0
    for T in (100, 300, 2047):
        x, w = operands(T, 4064, 200, "e4m3", 1, gpu)
        a, s = product(x, w, "e4m3", ws_fill=0xFF)
        b, _ = product(x, w, "e4m3", ws_fill=0)
        assert torch.equal(a, b)
        used += B.mx_linear_workspace_bytes(s) > 0
    assert used


def test_prepared_layout(gpu):
    """The tiled weights against their documented formula."""
    K, N = 160, 70
    g = gen(9)
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    sf = torch.randint(0, 255, (N, K // 32), generator=g, dtype=torch.uint8)
    t = B.mx_linear_prepare(B.make_mx_linear(1, K, N), w.to(gpu), sf.to(gpu)).cpu()
    blocks, KT = 2 * ((N + 63) // 64), (K + 127) // 128
    codes, scales = t[:blocks * KT * 2048].view(blocks, KT, 128, 16), t[blocks * KT * 2048:].view(blocks, KT, 32, 4)
    for b, kt, p in itertools.product(range(blocks), range(KT), range(128)):
        c = p >> 2
        n, k = 64 * (b // 2) + 2 * c + b % 2, 128 * kt + 32 * ((p & 3) ^ ((c >> 2) & 3))
        want = w[n, k // 2:k // 2 + 16] if n < N and k < K else torch.zeros(16, dtype=torch.uint8)
        assert torch.equal(codes[b, kt, p], want)
    for b, kt, c, j in itertools.product(range(blocks), range(KT), range(32), range(4)):
        n, k = 64 * (b // 2) + 2 * c + b % 2, 4 * kt + j
        assert scales[b, kt, c, j] == (sf[n, k] if n < N and k < K // 32 else 0)
