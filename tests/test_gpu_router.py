"""GPU parity of moe_router_logits.

Small whole numbers make every product and partial sum exact in FP32, in any order, so those results are
compared bit for bit.  Random operands are held to the worst case of an FP32 sum of n products in any order,
n * 2^-23 of the sum of their magnitudes (2^-23: a sum inside a matrix instruction may truncate).
"""
import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def run(x, w, T=None, shape=None, fill=0x5A):
    T = x.shape[0]
    E, H = w.shape
    s = shape or B.make_router(T, H, E, weight_dtype=w.dtype)
    logits = torch.full((T, E), float("nan"), dtype=F32, device=x.device)
    ws = torch.full((B.router_workspace_bytes(s),), fill, dtype=torch.uint8, device=x.device)
    B.router_logits(s, x, B.router_prepare(s, w), logits, ws)
    torch.cuda.synchronize()
    return logits


def whole(T, H, E, wt, seed, device):
    """Operands whose sums stay below 2^24: |x| <= 15, |w| <= 3 (BF16) or up to 2^11 on few columns (FP32)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-15, 16, (T, H), generator=g).float()
    w = torch.randint(-3, 4, (E, H), generator=g).float()
    if wt == F32:   # more than 8 significant bits on every 61st column, so that the parts all take part
        w[:, ::61] = torch.randint(-1500, 1501, (E, (H + 60) // 61), generator=g).float()
    assert (x.abs().sum(1).max() * 3 + 15 * 1500 * (H // 61 + 1)) < 2 ** 24
    return x.to(BF16).to(device), w.to(wt).to(device)


# T around every tile edge, E that fill no tile, one K-step to long rows
SIZES = [(1, 32, 1), (1, 7168, 256), (3, 64, 8), (16, 96, 16), (17, 4096, 64), (31, 1056, 100), (64, 7168, 384),
         (65, 2048, 257), (127, 7168, 256), (128, 7168, 256), (129, 512, 512), (200, 4096, 1000), (255, 32, 1024),
         (1000, 992, 77), (513, 7168, 129), (2047, 4096, 64), (4097, 1024, 255), (9000, 480, 48), (33000, 64, 40)]


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("T,H,E", SIZES)
def test_router_exact(gpu, T, H, E, wt):
    print(f"router T={T} H={H} E={E} {wt}", flush=True)
    x, w = whole(T, H, E, wt, T + E, gpu)
    got = run(x, w)
    want = x.double() @ w.double().t().contiguous()
    assert torch.equal(got.double(), want)


# every tile shape, whole and with ragged tokens, experts and columns, in one piece and split
TILES = [(257, 1056, 256), (600, 4128, 256), (1500, 2080, 100), (3000, 480, 60), (4200, 7168, 64), (8191, 288, 256),
         (8300, 96, 200), (8300, 160, 300), (9000, 1120, 257), (16400, 160, 128), (16385, 64, 385), (20000, 96, 512),
         (70000, 32, 64), (60000, 96, 300), (65000, 32, 257), (65536, 160, 384)]


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("T,H,E", TILES)
def test_router_exact_tiles(gpu, T, H, E, wt):
    print(f"router T={T} H={H} E={E} {wt}", flush=True)
    x, w = whole(T, H, E, wt, T + E, gpu)
    got = run(x, w)
    want = x.double() @ w.double().t().contiguous()
    assert torch.equal(got.double(), want)


# the tiles of the larger shapes again with a split and without, ragged in every direction; many rows of 16-token tiles
PIECES = [(40, 20000, 860), (130, 1056, 100), (1024, 1056, 40), (1100, 4128, 200), (1300, 7136, 257), (1030, 2080, 520),
          (2100, 7136, 300), (4100, 4064, 500), (3100, 7136, 380), (17000, 2080, 250), (3000, 4128, 120)]


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("T,H,E", PIECES)
def test_router_exact_pieces(gpu, T, H, E, wt):
    print(f"router T={T} H={H} E={E} {wt}", flush=True)
    x, w = whole(T, H, E, wt, T + E, gpu)
    got = run(x, w)
    want = x.double() @ w.double().t().contiguous()
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("T,H,E", [(1, 7168, 256), (130, 7168, 256), (700, 4096, 64), (5000, 1024, 384)])
def test_router_random(gpu, T, H, E, wt):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, H, generator=g).to(BF16).to(gpu)
    w = (torch.randn(E, H, generator=g) / H ** 0.5).to(wt).to(gpu)
    got = run(x, w).double()
    xd, wd = x.double(), w.double().t().contiguous()
    n = H * (3 if wt == F32 else 1)
    assert ((got - xd @ wd).abs() <= n * 2.0 ** -23 * (xd.abs() @ wd.abs())).all()


def test_router_f32_weights_keep_all_bits(gpu):
    """A row of x that picks one column returns that column of the weights, bit for bit."""
    H, E = 128, 37
    w = torch.randn(E, H, generator=torch.Generator().manual_seed(6)) * torch.exp2(torch.arange(H) % 60 - 30.0)
    got = run(torch.eye(H).to(BF16).to(gpu), w.to(gpu))
    assert torch.equal(got, w.t().contiguous().to(gpu))


def test_router_rows(gpu):
    """Strided rows of x, an x that ends where its memory ends, and rows of logits behind the last."""
    x, w = whole(50, 256, 33, BF16, 9, gpu)
    want = run(x, w)
    wide = torch.full((50, 320), float("nan"), dtype=BF16, device=gpu)
    wide[:, :256] = x
    got = run(wide[:, :256], w, shape=B.make_router(50, 256, 33, x_stride=320))
    assert torch.equal(got, want)
    s = B.make_router(20, 256, 33)
    logits = torch.full((50, 33), 4.0, device=gpu)
    ws = torch.empty(B.router_workspace_bytes(s), dtype=torch.uint8, device=gpu)
    B.router_logits(s, x[:20], B.router_prepare(s, w), logits[:20], ws)
    torch.cuda.synchronize()
    assert torch.equal(logits[:20], want[:20]) and (logits[20:] == 4.0).all()


@pytest.mark.parametrize("T", [1, 40, 300, 3000])
def test_router_same_for_a_row_alone_and_again(gpu, T):
    """Bit-identical from call to call, whatever the workspace holds."""
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(T, 7168, generator=g).to(BF16).to(gpu), torch.randn(256, 7168, generator=g).to(BF16).to(gpu)
    a = run(x, w)
    for fill in (0x00, 0xFF):
        assert torch.equal(a, run(x, w, fill=fill))


def test_router_nan_rows_stay_apart(gpu):
    x, w = whole(40, 512, 20, BF16, 10, gpu)
    want = run(x, w)
    x[7, 3], x[21, 500] = float("nan"), float("inf")
    got = run(x, w)
    keep = torch.ones(40, dtype=torch.bool)
    keep[[7, 21]] = False
    assert torch.isnan(got[7]).all() and not torch.isfinite(got[21]).any()
    assert torch.equal(got[keep.to(gpu)], want[keep.to(gpu)])


@pytest.mark.parametrize("T", [5, 40, 3000])
def test_router_infinite_x_with_f32_weights(gpu, T):
    """A row with an infinity has no finite logit where its weight is not 0; the other rows keep theirs."""
    x, w = whole(T, 512, 20, F32, 11, gpu)
    w[:, 500] = torch.where(w[:, 500] == 0, 1.0, w[:, 500])
    want = run(x, w)
    x[3, 500] = float("inf")
    got = run(x, w)
    assert not torch.isfinite(got[3]).any()
    keep = torch.arange(T, device=gpu) != 3
    assert torch.equal(got[keep], want[keep])


def test_router_graphs_share_a_workspace(gpu):
    """Two captured products over one workspace of partial sums, replayed in turn on one stream with eager
    products of the same workspace between them."""
    (T, E, H), n = (300, 256, 4096), 2
    shapes = [B.make_router(T, H, E, weight_dtype=wt) for wt in (BF16, F32)]
    sizes = [B.router_workspace_bytes(s) for s in shapes]
    assert min(sizes) > 0
    ws = torch.full((max(sizes),), 0x5A, dtype=torch.uint8, device=gpu)
    ops = [whole(T, H, E, wt, 12 + i, gpu) for i, wt in enumerate((BF16, F32))]
    tiled = [B.router_prepare(s, w) for s, (_, w) in zip(shapes, ops)]
    out = [torch.empty(T, E, device=gpu) for _ in range(n)]
    graphs = []
    for s, (x, _), t, o in zip(shapes, ops, tiled, out):
        B.router_logits(s, x, t, o, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.router_logits(s, x, t, o, ws)
        graphs.append(graph)
    for seed in (20, 21, 22):
        for i, wt in enumerate((BF16, F32)):
            ops[i][0].copy_(whole(T, H, E, wt, seed + 10 * i, gpu)[0])
        eager = torch.empty(T, E, device=gpu)
        for o in out:
            o.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        B.router_logits(shapes[0], ops[0][0], tiled[0], eager, ws)
        torch.cuda.synchronize()
        for (x, w), o in zip(ops, out):
            assert torch.equal(o.double(), x.double() @ w.double().T)
        assert torch.equal(eager, out[0])


def test_router_no_tokens(gpu):
    s = B.make_router(0, 64, 8)
    w = torch.ones(8, 64, dtype=BF16, device=gpu)
    x = torch.zeros(0, 64, dtype=BF16, device=gpu)
    B.router_logits(s, x, B.router_prepare(s, w), torch.zeros(0, 8, device=gpu))


def test_router_binding_refusals(gpu):
    x, w = whole(20, 64, 8, BF16, 11, gpu)
    s = B.make_router(20, 64, 8)
    wt, out = B.router_prepare(s, w), torch.empty(20, 8, device=gpu)
    for a in ((x[:19], wt, out), (x.float(), wt, out), (x, wt[:-16], out), (x, w, out), (x, wt, out[:, :7]),
              (x, wt, out.half()), (x.cpu(), wt, out), (x, wt, out.cpu())):
        with pytest.raises((TypeError, ValueError)):
            B.router_logits(s, *a)
    with pytest.raises(TypeError):
        B.router_prepare(s, w.float())
    with pytest.raises(ValueError):
        B.router_prepare(s, w[:7])


@pytest.mark.parametrize("wt", [BF16, F32])
def test_router_more_rows_than_a_launch(gpu, wt):
    """Over 2^24 tokens, strided; sums of small whole numbers, so FP32 products of any order are exact too."""
    T, H, E = (1 << 24) + 3001, 32, 20
    g = torch.Generator(device=gpu).manual_seed(30)
    wide = torch.randint(-15, 16, (T, 40), generator=g, device=gpu, dtype=torch.int8).to(BF16)
    w = torch.randint(-3, 4, (E, H), generator=g, device=gpu).to(wt)
    got = run(wide[:, :H], w, shape=B.make_router(T, H, E, weight_dtype=wt, x_stride=40))
    for rows in (slice(0, 5000), slice((1 << 24) - 5000, T)):
        assert torch.equal(got[rows], wide[rows, :H].float() @ w.float().t().contiguous())
    both = w.float().sum(0)
    for x, l in zip(wide.split(1 << 22), got.split(1 << 22)):    # (the library's product with a vector stops at 2^24 rows)
        assert torch.equal(l.sum(1), (x[:, :H].float() * both).sum(1))


@pytest.mark.parametrize("wt", [BF16, F32])
def test_router_one_workspace_for_all_batches(gpu, wt):
    """A workspace of the largest batch serves the smaller ones, of which some need more than the largest."""
    H, E, most = 7168, 256, 20000
    x, w = whole(most, H, E, wt, 31, gpu)
    want = x.double() @ w.double().t().contiguous()
    shape = B.make_router(most, H, E, weight_dtype=wt)
    tiled = B.router_prepare(shape, w)
    ws = torch.full((B.router_max_workspace_bytes(shape),), 0x5A, dtype=torch.uint8, device=gpu)
    own = []
    for T in (most, 1, 33, 128, 300, 512, 1000, 2048, 4096, 8192, 16384):
        s = B.make_router(T, H, E, weight_dtype=wt)
        own.append(B.router_workspace_bytes(s))
        logits = torch.full((T, E), float("nan"), device=gpu)
        B.router_logits(s, x[:T], tiled, logits, ws)
        assert torch.equal(logits.double(), want[:T])
    assert max(own) > 0


# FP32 weights in every tile, whole and split, on runs of columns that do and do not fill the last step
F32_TILES = [((16, 16), False, 100, 480, 40), ((16, 16), False, 20, 96, 8), ((32, 64), False, 1500, 480, 40),
             ((32, 64), True, 20, 7136, 200), ((64, 64), False, 9000, 96, 40), ((64, 64), False, 2100, 480, 200),
             ((64, 64), True, 300, 4128, 257), ((64, 64), True, 700, 2080, 100), ((64, 128), False, 4200, 480, 200),
             ((64, 128), True, 700, 7136, 200), ((64, 128), True, 1100, 4128, 257), ((128, 128), False, 9000, 480, 200),
             ((128, 128), True, 1100, 7136, 257), ((128, 128), True, 4200, 2080, 200)]


def without(w, part):
    """FP32 weights less one of their three parts of 8 bits."""
    parts, rest = [], w.clone()
    for _ in range(3):
        parts.append((rest.view(torch.int32) & -65536).view(F32))
        rest = rest - parts[-1]
    assert not rest.any()
    return w - parts[part]


@pytest.mark.parametrize("tile,split,T,H,E", F32_TILES)
def test_router_f32_weights_keep_all_parts(gpu, tile, split, T, H, E):
    """Weights of 24 bits, one column to a row of x; then whole numbers of 20 bits, 15 columns to a row, whose sums stay
    below 2^24.  Without any one of the parts nearly no logit is right."""
    got_tile = B.router_tile(B.make_router(T, H, E, weight_dtype=F32))
    print(f"router T={T} H={H} E={E} tile {got_tile}", flush=True)
    assert got_tile[:2] == tile and (got_tile[2] > 1) == split
    g = torch.Generator().manual_seed(T + H + E)
    one = torch.zeros(T, H, dtype=BF16)
    one[torch.arange(T), torch.randperm(max(T, H), generator=g)[:T] % H] = 1
    bits24 = torch.randn(E, H, generator=g) * torch.exp2(torch.arange(H) % 60 - 30.0)
    few = torch.zeros(T, H, dtype=BF16)
    few.scatter_(1, torch.rand(T, H, generator=g).topk(15, dim=1).indices, 1)
    whole20 = torch.randint(-2 ** 20 + 1, 2 ** 20, (E, H), generator=g).float()
    for x, w in ((one, bits24), (few, whole20)):
        want = x.double() @ w.double().t().contiguous()
        assert torch.equal(run(x.to(gpu), w.to(gpu)).cpu().double(), want)
        for part in range(3):
            rows = x[:200].double() @ without(w, part).double().t().contiguous()
            assert (rows != want[:200]).float().mean() > 0.8
