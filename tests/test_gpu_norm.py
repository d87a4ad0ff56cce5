"""GPU parity of moe_norm_quant against the float64 oracle.

Tolerances.  v carries at most four FP32 roundings (h, rsqrt's result, two products): 4 * 2^-24 relative; y adds
BF16's 2^-8, residual_out one FP32 and one BF16 rounding; an E4M3 code is off by at most half a step, 2^-4 relative
or 2^-10 below the smallest normal value.  Scale codes are equal.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B
from oracle.front import norm_ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
V_REL = 4 * 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: 0.0}


def f64(t):
    return t.double().cpu().numpy()


def values(codes):
    return codes.view(torch.float8_e4m3fn).float().double().cpu().numpy()


def draw(T, H, xt, rt, wt, seed, device):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g) * torch.exp2(torch.randint(-6, 7, (T, 1), generator=g).float())
    x *= torch.exp2(torch.randint(-3, 4, (H,), generator=g).float())
    w = 1 + 0.3 * torch.randn(H, generator=g)
    r = None if rt is None else torch.randn(T, H, generator=g).to(rt).to(device)
    return x.to(xt).to(device), r, w.to(wt).to(device)


def check(out, x, r, w, eps):
    h, v, code, scaled = norm_ref(f64(x), f64(w), eps, None if r is None else f64(r))
    T, H = v.shape
    if "residual_out" in out:
        tol = np.abs(h) * (2.0 ** -24 + HALF[out["residual_out"].dtype] * (1 + 2.0 ** -24))
        assert (np.abs(f64(out["residual_out"]) - h) <= tol).all()
    if "y" in out:
        assert (np.abs(f64(out["y"]) - v) <= np.abs(v) * (2.0 ** -8 + 1.01 * V_REL) + 2.0 ** -133).all()
    if "x_q" in out:
        assert np.array_equal(out["x_sf"].cpu().numpy(), code)
        tol = np.maximum(2.0 ** -4 * np.abs(scaled), 2.0 ** -10) + 1.1 * V_REL * np.abs(scaled)
        assert (np.abs(values(out["x_q"]) - scaled) <= tol).all()


def run(x, r, w, eps=1e-6, rt=None, outs=("y", "q", "r"), rout=None, shape=None):
    T, H = x.shape
    rt = rt or (BF16 if r is None else r.dtype)
    s = shape or B.make_norm(T, H, eps, x.dtype, rt, w.dtype)
    out = {}
    if "y" in outs:
        out["y"] = torch.full((T, H), float("nan"), dtype=BF16, device=x.device)
    if "q" in outs:
        out["x_q"] = torch.full((T, H), 0x55, dtype=torch.uint8, device=x.device)
        out["x_sf"] = torch.full((T, H // 32), 0x55, dtype=torch.uint8, device=x.device)
    if "r" in outs:
        out["residual_out"] = torch.full((T, H), float("nan"), dtype=rt, device=x.device) if rout is None else rout
    B.norm_quant(s, x, w, residual=r, **out)
    torch.cuda.synchronize()
    return out


# one row to many, one block of columns to the largest rows, odd multiples of 32, every vector and row split
SIZES = [(1, 32), (5, 64), (3, 96), (257, 256), (2, 480), (7, 512), (3, 544), (33, 2048), (1, 7168), (130, 7168),
         (9, 4096), (3, 8160), (5, 8192), (2, 16384), (3, 20000), (2, 32768), (2, 32800), (1, 65536), (1, 1 << 20)]


@pytest.mark.parametrize("T,H", SIZES)
def test_norm_sizes(gpu, T, H):
    print(f"norm T={T} H={H}", flush=True)
    x, r, w = draw(T, H, BF16, BF16, BF16, T + H, gpu)
    check(run(x, r, w), x, r, w, 1e-6)


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("rt", [None, BF16, F32])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_norm_types_and_outputs(gpu, xt, rt, wt):
    for i, (T, H) in enumerate([(6, 352), (5, 7168), (2, 33024)]):
        x, r, w = draw(T, H, xt, rt, wt, i, gpu)
        full = run(x, r, w, eps=1e-3)
        check(full, x, r, w, 1e-3)
        for outs in (("y",), ("q",), ("y", "q"), ("q", "r"), ("y", "r")):
            part = run(x, r, w, eps=1e-3, outs=outs)
            for k, t in part.items():
                assert torch.equal(t.view(torch.uint8), full[k].view(torch.uint8)), (outs, k)


@pytest.mark.parametrize("H", [64, 1024, 7168, 40960])
def test_norm_in_place(gpu, H):
    """residual_out may be the residual, or x."""
    x, r, w = draw(19, H, BF16, BF16, BF16, 7, gpu)
    want = run(x, r, w)
    for alias in ("residual", "x"):
        x2, r2 = x.clone(), r.clone()
        got = run(x2, r2, w, rout=r2 if alias == "residual" else x2)
        for k in want:
            assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), (alias, k)


@pytest.mark.parametrize("T,H", [(7, 32), (31, 64), (33, 96), (17, 128), (1000, 160), (9, 192), (63, 224), (4099, 256)])
def test_norm_short_rows(gpu, T, H):
    """Rows that share a wave: ragged counts, strides, in place, nothing behind the last row."""
    x, r, w = draw(T, H, F32, BF16, F32, 22, gpu)
    want = run(x, r, w)
    check(want, x, r, w, 1e-6)
    rs = torch.full((T + 40, H + 8), 9.0, dtype=BF16, device=gpu)
    rs[:T, :H] = r
    y = torch.full((T + 40, H), 5.0, dtype=BF16, device=gpu)
    q = torch.full((T + 40, H), 0x11, dtype=torch.uint8, device=gpu)
    sf = torch.full((T + 40, H // 32), 0x22, dtype=torch.uint8, device=gpu)
    s = B.make_norm(T, H, 1e-6, F32, BF16, F32, residual_stride=H + 8, residual_out_stride=H + 8)
    B.norm_quant(s, x, w, q[:T], sf[:T], y=y[:T], residual=rs[:T, :H], residual_out=rs[:T, :H])
    torch.cuda.synchronize()
    for got, k in ((y[:T], "y"), (q[:T], "x_q"), (sf[:T], "x_sf"), (rs[:T, :H], "residual_out")):
        assert torch.equal(got, want[k]), k
    assert (y[T:] == 5.0).all() and (q[T:] == 0x11).all() and (sf[T:] == 0x22).all()
    assert (rs[T:] == 9.0).all() and (rs[:, H:] == 9.0).all()


def test_norm_strides(gpu):
    """Rows of wider buffers; what lies between them stays as it is."""
    T, H = 11, 608
    x, r, w = draw(T, H, BF16, F32, F32, 8, gpu)
    want = run(x, r, w)
    xs = torch.full((T, 640), 7.0, dtype=BF16, device=gpu)
    rs, ro = (torch.full((T, 616), 9.0, dtype=F32, device=gpu), torch.full((T, 800), 3.0, dtype=F32, device=gpu))
    xs[:, :H], rs[:, :H] = x, r
    s = B.make_norm(T, H, 1e-6, BF16, F32, F32, x_stride=640, residual_stride=616, residual_out_stride=800)
    got = run(xs[:, :H], rs[:, :H], w, shape=s, rt=F32, rout=ro[:, :H])
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert (ro[:, H:] == 3.0).all() and (xs[:, H:] == 7.0).all()


def test_norm_more_rows_than_a_grid_axis(gpu):
    """Over 2^20 rows; rows do not depend on where they lie, so the ends are compared with calls of their own."""
    T, H = (1 << 20) + 5, 32
    g = torch.Generator(device=gpu).manual_seed(21)
    x = torch.randn(T, H, generator=g, device=gpu).to(BF16)
    r = torch.randn(T, H, generator=g, device=gpu).to(BF16)
    w = (1 + 0.3 * torch.randn(H, generator=g, device=gpu)).to(BF16)
    got = run(x, r, w)
    h = x.float() + r.float()
    v = h.double() / torch.sqrt(h.double().square().mean(1, keepdim=True) + 1e-6) * w.double()
    assert ((got["y"].double() - v).abs() <= v.abs() * (2.0 ** -8 + 1.01 * V_REL) + 2.0 ** -133).all()
    for rows in (slice(0, 40), slice((1 << 20) - 20, T)):
        alone = run(x[rows], r[rows], w)
        check(alone, x[rows], r[rows], w, 1e-6)
        for k in alone:
            assert torch.equal(alone[k], got[k][rows]), k


def test_norm_rows_behind_the_last_stay(gpu):
    x, r, w = draw(8, 7168, BF16, BF16, BF16, 9, gpu)
    y = torch.full((8, 7168), 5.0, dtype=BF16, device=gpu)
    q = torch.full((8, 7168), 0x11, dtype=torch.uint8, device=gpu)
    sf = torch.full((8, 224), 0x22, dtype=torch.uint8, device=gpu)
    B.norm_quant(B.make_norm(3, 7168), x[:3], w, q[:3], sf[:3], y[:3], r[:3])
    torch.cuda.synchronize()
    assert (y[3:] == 5.0).all() and (q[3:] == 0x11).all() and (sf[3:] == 0x22).all()
    assert not (y[:3] == 5.0).all()


@pytest.mark.parametrize("H", [32, 224, 7168])
def test_norm_scale_border(gpu, H):
    """Blocks whose maximum lies on 448 * 2^s, or a few FP32 steps to either side, of the formula in 64 bits."""
    g = torch.Generator().manual_seed(H)
    codes = set()
    for _ in range(max(2, 6000 // H)):
        x = torch.randn(1, H, generator=g)
        x[0, 31::32] = x[0, 31::32].abs() + 0.5
        w = torch.full((H,), 0.25)
        # the weight of every 32nd column brings its v to 3.5 (1 + a few 2^-24), above all others of its block
        rstd = 1 / (x.double().square().mean() + 1e-6).sqrt()
        step = 1 + torch.randint(-2, 3, (H // 32,), generator=g).double() * 2.0 ** -24
        w[31::32] = (3.5 * step / (x[0, 31::32].double() * rstd)).float()
        x, w = x.to(gpu), w.to(gpu)
        out = run(x, None, w, outs=("q", "y"))
        _, v, code, _ = norm_ref(f64(x), f64(w), 1e-6)
        assert (np.abs(v[:, 31::32] / 3.5 - 1) < 2.0 ** -20).all()
        codes |= set(code.ravel().tolist())
        check(out, x, None, w, 1e-6)
    assert codes == {120, 121}


def test_norm_small_and_large_values(gpu):
    for scale in (1e-30, 1e-10, 1e10, 1e30):
        x, r, w = draw(4, 1024, F32, F32, F32, 10, gpu)
        x, r = x * scale, r * scale
        check(run(x, r, w, eps=0.0), x, r, w, 0.0)
    # v far below 1: scale codes down to 0
    x, r, w = draw(4, 1024, F32, F32, F32, 11, gpu)
    w = w * torch.exp2(-torch.arange(32, device=gpu).repeat_interleave(32).float() * 4)
    out = run(x, r, w, outs=("q",))
    assert int(out["x_sf"].min()) == 0
    check(out, x, r, w, 1e-6)


def test_norm_zero_rows_and_blocks(gpu):
    x, r, w = draw(4, 96, BF16, None, BF16, 12, gpu)
    x[1] = 0
    x[2, 32:64] = 0
    out = run(x, r, w)
    check(out, x, r, w, 1e-6)
    assert (out["x_sf"][1] == 0).all() and (values(out["x_q"])[1] == 0).all() and (out["y"][1] == 0).all()
    out = run(x, r, w, eps=0.0)
    assert torch.isnan(out["y"][1]).all() and torch.isfinite(out["y"][0]).all()


def test_norm_nan_and_infinity(gpu):
    x, r, w = draw(3, 96, F32, None, F32, 13, gpu)
    x[0, 5], x[1, 40] = float("nan"), float("inf")
    out = run(x, r, w, rt=F32)
    y, q = out["y"].float().cpu(), values(out["x_q"])
    assert torch.isnan(y[0]).all() and np.isnan(q[0]).all()
    assert torch.isnan(y[1, 40]) and np.isnan(q[1, 40])
    assert (np.delete(q[1], 40) == 0).all() and torch.isfinite(y[2]).all()
    assert torch.isfinite(out["residual_out"][2]).all()


def test_norm_no_tokens(gpu):
    x = torch.zeros(0, 64, dtype=BF16, device=gpu)
    B.norm_quant(B.make_norm(0, 64), x, torch.ones(64, dtype=BF16, device=gpu), y=x)


def test_norm_binding_refusals(gpu):
    x, r, w = draw(4, 64, BF16, BF16, BF16, 14, gpu)
    y, s = torch.empty_like(x), B.make_norm(4, 64)
    for kw in (dict(y=y[:3]), dict(y=y.float()), dict(y=y, residual=r.float()), dict(y=y, residual=r.cpu()),
               dict(y=y, residual=r.t()), dict(y=y, residual_out=y[:, ::2])):
        with pytest.raises((TypeError, ValueError)):
            B.norm_quant(s, x, w, **kw)
    with pytest.raises(ValueError):
        B.norm_quant(s, x, w[:32], y=y)
    with pytest.raises(B.MoeError):
        B.norm_quant(s, x, w)
    with pytest.raises(B.MoeError):
        B.norm_quant(B.make_norm(4, 48), x[:, :48].contiguous(), w[:48], y=y[:, :48].contiguous())


@pytest.mark.parametrize("xt", [F32, BF16])
def test_norm_scale_border_of_sums(gpu, xt):
    """Rows whose FP32 sums x + residual are rounded, and whose largest v lies between what the rounded and the whole
    sums give for 448 * 2^s: the scale is that of the whole sums."""
    H, found = 32, 0
    g = torch.Generator().manual_seed(77)
    for _ in range(1500):
        x, r = torch.randn(1, H, generator=g).to(xt), 4 * torch.randn(1, H, generator=g)
        w = torch.full((H,), 0.25)
        whole, rounded = x.double() + r.double(), (x.float() + r).double()
        rstd = [1 / (h.square().mean() + 1e-6).sqrt() for h in (whole, rounded)]
        w[31] = (3.5 / (whole[0, 31].abs() * (rstd[0] + rstd[1]) / 2)).float()
        v = [(whole[0, 31].abs() * s * w[31].double()).item() / 3.5 - 1 for s in rstd]
        if (v[0] > 0) == (v[1] > 0) or abs(v[0]) < 2.0 ** -40:   # 3.5 in both, or no clear side
            continue
        found += 1
        x, r, w = x.to(gpu), r.to(gpu), w.to(gpu)
        check(run(x, r, w), x, r, w, 1e-6)
    assert found >= 20


@pytest.mark.parametrize("H", [64, 2048, 40960])
def test_norm_sums_beyond_fp32(gpu, H):
    """x + residual over FP32's range is an infinity as any other: NaN at its place, 0 in the rest of its row."""
    x, r, w = draw(5, H, F32, F32, F32, 16, gpu)
    x[1, H - 2], r[1, H - 2] = 3e38, 3e38
    x[2, 3], r[2, 3] = -3e38, -2e38
    x[3, 5], r[3, 5] = 3e38, 3e37           # 3.3e38 is inside
    x[4, 7], r[4, 7] = 3e38, -3e38
    out = run(x, r, w)
    y, q = out["y"].float().cpu(), values(out["x_q"])
    for t, c in ((1, H - 2), (2, 3)):
        assert torch.isinf(out["residual_out"][t, c]) and torch.isnan(y[t, c]) and np.isnan(q[t, c])
        assert (np.delete(y[t].numpy(), c) == 0).all() and (np.delete(q[t], c) == 0).all()
    keep = [0, 3, 4]
    check({k: v[keep] for k, v in out.items()}, x[keep], r[keep], w, 1e-6)


@pytest.mark.parametrize("power", [-140, -130, -120, -70, 70, 110, 124])
def test_norm_far_from_one_without_eps(gpu, power):
    """Rows whose 1 / rms FP32 does not hold, or not in full: sizes, and blocks on a border of the scale."""
    for rt in (None, F32):
        x, r, w = draw(4, 1024, F32, rt, F32, 15, gpu)
        x = torch.ldexp(x.clamp(-4, 4), torch.tensor(power))
        r = None if r is None else torch.ldexp(r.clamp(-4, 4), torch.tensor(power))
        check(run(x, r, w, eps=0.0, rt=F32), x, r, w, 0.0)
    g = torch.Generator().manual_seed(power + 200)
    codes, H = set(), 224
    for _ in range(40):
        x = torch.ldexp(torch.randn(1, H, generator=g).clamp(-4, 4), torch.tensor(power))
        x[0, 31::32] = x[0, 31::32].abs() + 2.0 ** (power - 1)
        w = torch.full((H,), 0.25)
        rstd = 1 / x.double().square().mean().sqrt()
        step = 1 + torch.randint(-2, 3, (H // 32,), generator=g).double() * 2.0 ** -24
        w[31::32] = (3.5 * step / (x[0, 31::32].double() * rstd)).float()
        x, w = x.to(gpu), w.to(gpu)
        out = run(x, None, w, eps=0.0, rt=F32, outs=("q", "y"))
        codes |= set(norm_ref(f64(x), f64(w), 0.0)[2].ravel().tolist())
        check(out, x, None, w, 0.0)
    assert codes == {120, 121}


def test_norm_one_row_in_place_of_any_stride(gpu):
    """A single row has no next one for a stride to say anything about."""
    x, r, w = draw(1, 512, BF16, BF16, BF16, 17, gpu)
    want = run(x, r, w)
    got = run(x, r, w, rout=r, shape=B.make_norm(1, 512, x_stride=512, residual_stride=1024, residual_out_stride=520))
    for k in want:
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k
