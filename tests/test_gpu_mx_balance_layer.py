"""Quantisation, the dense product, the balance of the load and the gate's gradient run together as a layer uses them:
the experts' weights quantised here and streamed by the forward, a shared expert in 4 bits beside them, the gate's choice
counted, and the gradient back at the logits; eager, on side streams, bound and as replays of graphs."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B
from moe_expert_ffn_plan_amd import inputs
from oracle.balance import balance_ref, gate_grad_ref
from oracle.formats import E2M1_TABLE, E4M3_TABLE
from oracle.forward import forward_ref
from oracle.mx import mx_quant_ref
from parity import assert_y_gate

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
T, H, I, E, K, S = 200, 512, 256, 16, 4, 3
W = inputs.Workload("beside", T, H, I, E, E, K, 16, "uniform", seed=43, weight_seed=53)


def u8(dev, *s, fill=0xA5):
    return torch.full(s, fill, dtype=torch.uint8, device=dev)


class Layer:
    """Weights, plans and buffers of the layer, and its calls in order."""

    def __init__(self, dev, seed=0):
        g = torch.Generator().manual_seed(60 + seed)
        self.dev = dev
        self.w1 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).to(dev)
        self.w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).to(dev)
        self.sw1 = (torch.randn(2 * I, H, generator=g) / H ** 0.5).to(dev)
        self.router = (torch.randn(E, H, generator=g) / H ** 0.5).to(BF16).to(dev)
        self.plain = {}
        for name, w in (("w1", self.w1), ("w2", self.w2)):
            q, sf = u8(dev, E * w.shape[1], w.shape[2] // 2), u8(dev, E * w.shape[1], w.shape[2] // 32)
            B.mx_quant(B.make_mx_quant(E * w.shape[1], w.shape[2], "e2m1", F32), w.view(-1, w.shape[2]), q, sf)
            self.plain[name], self.plain[name + "_sf"] = q, sf
        self.moe = B.shape_of(W)
        self.tiled = B.prepare_all(self.moe, self.plain)
        self.shared_q, self.shared_sf = u8(dev, 2 * I, H // 2), u8(dev, 2 * I, H // 32)
        B.mx_quant(B.make_mx_quant(2 * I, H, "e2m1", F32), self.sw1, self.shared_q, self.shared_sf)
        self.lin4 = B.make_mx_linear(T, H, 2 * I, "e2m1")
        self.lin8 = B.make_mx_linear(T, H, 2 * I, "e4m3")
        self.shared = B.mx_linear_prepare(self.lin4, self.shared_q, self.shared_sf)
        self.quant = B.make_mx_quant(T, H, "e2m1")
        self.norm, self.norm_w = B.make_norm(T, H), torch.ones(H, dtype=BF16, device=dev)
        self.rt = B.make_router(T, H, E)
        self.router_t = B.router_prepare(self.rt, self.router)
        self.gate = B.make_gate(T, E, K, scale=1.5)
        self.bal = B.make_balance(T, E, K, num_seqs=S, scale=1.5)
        self.off = torch.tensor([0, 90, 90, 180], device=dev)
        self.x_q, self.x_sf, self.q4, self.sf4 = u8(dev, T, H), u8(dev, T, H // 32), u8(dev, T, H // 2), u8(dev, T, H // 32)
        self.y = torch.empty(T, H, dtype=BF16, device=dev)
        self.logits = torch.empty(T, E, device=dev)
        self.ids, self.w = torch.empty(T, K, dtype=torch.int64, device=dev), torch.empty(T, K, device=dev)
        self.out = torch.empty(T, H, dtype=BF16, device=dev)
        self.up4, self.up8 = (torch.empty(T, 2 * I, dtype=BF16, device=dev) for _ in range(2))
        self.counts = torch.empty(S, E, dtype=torch.int32, device=dev)
        self.rows = torch.empty(S, dtype=torch.int32, device=dev)
        self.share, self.loss, self.z = torch.empty(S, E, device=dev), torch.empty(S, device=dev), torch.empty(S, device=dev)
        self.d_loss, self.d_z = torch.tensor([0.5, 1.0, 2.0], device=dev), torch.tensor([0.1, 0.2, 0.3], device=dev)
        self.d_w = (torch.randn(T, K, generator=g) / T).to(dev)
        self.d_logits = torch.zeros(T, E, device=dev)
        self.ws = u8(dev, B.forward_workspace_bytes(self.moe))
        self.rws = u8(dev, B.router_workspace_bytes(self.rt))
        self.lws = u8(dev, max(B.mx_linear_workspace_bytes(s) for s in (self.lin4, self.lin8)))
        self.bws = u8(dev, B.balance_workspace_bytes(self.bal))

    def calls(self, x, **kw):
        t = self.tiled
        return [B.norm_quant(self.norm, x, self.norm_w, self.x_q, self.x_sf, self.y, **kw),
                B.router_logits(self.rt, self.y, self.router_t, self.logits, self.rws, **kw),
                B.gate(self.gate, self.logits, self.ids, self.w, **kw),
                B.balance(self.bal, self.logits, self.ids, self.bws, seq_offsets=self.off, counts=self.counts, rows=self.rows,
                          share=self.share, loss=self.loss, z=self.z, **kw),
                B.forward(self.moe, self.x_q, self.x_sf, self.ids, self.w, t["w1"], t["w1_sf"], t["w2"], t["w2_sf"], self.out,
                          self.ws, **kw),
                B.mx_quant(self.quant, self.y, self.q4, self.sf4, **kw),
                B.mx_linear(self.lin4, self.q4, self.sf4, self.shared, self.up4, self.lws, **kw),
                B.mx_linear(self.lin8, self.x_q, self.x_sf, self.shared, self.up8, self.lws, **kw),
                B.gate_grad(self.bal, self.logits, self.ids, self.d_logits, seq_offsets=self.off, counts=self.counts,
                            rows=self.rows, d_loss=self.d_loss, d_z=self.d_z, d_topk_w=self.d_w, **kw)]

    def results(self):
        return [t.clone() for t in (self.out, self.up4, self.up8, self.counts, self.rows, self.share, self.loss, self.z, self.d_logits)]

    def spoil(self):
        for t in (self.out, self.up4, self.up8, self.counts, self.rows, self.share, self.loss, self.z, self.d_logits):
            t.view(torch.uint8).fill_(0x3C)
        for t in (self.ws, self.rws, self.lws, self.bws, self.q4, self.sf4, self.x_q):
            t.fill_(0xC3)
        self.d_logits[180:] = 0


def draw(dev, seed):
    return (3 * torch.randn(T, H, generator=torch.Generator().manual_seed(seed))).to(BF16).to(dev)


def same(a, b):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


def test_layer_against_the_oracle(gpu):
    L = Layer(gpu)
    L.calls(draw(gpu, 1))
    torch.cuda.synchronize()
    # the experts' weights as this library quantised them are the forward's
    for name, w in (("w1", L.w1), ("w2", L.w2)):
        codes, scales, _ = mx_quant_ref(w.view(-1, w.shape[2]).double().cpu().numpy(), "e2m1")
        assert np.array_equal(L.plain[name + "_sf"].cpu().numpy(), scales)
        assert np.array_equal(L.plain[name].cpu().numpy(), codes[:, 0::2] | codes[:, 1::2] << 4)
    d = {k: v.cpu().numpy().reshape(E, *s) for (k, v), s in zip(L.plain.items(), [(2 * I, H // 2), (2 * I, H // 32), (H, I // 2), (H, I // 32)])}
    ref = forward_ref(L.x_q.cpu().numpy(), L.x_sf.cpu().numpy(), L.ids.cpu().numpy(), L.w.cpu().numpy(), d["w1"], d["w1_sf"], d["w2"], d["w2_sf"],
                      num_experts=E, expert_begin=0, block_m=W.block_m)
    assert_y_gate(L.out.float().cpu().numpy(), ref["y"])
    # the shared expert's product from both formats, within BF16's rounding and the sums' own (2^-13 of the magnitudes)
    wv = np.ldexp(E2M1_TABLE[np.stack([d2 := L.shared_q.cpu().numpy() & 15, L.shared_q.cpu().numpy() >> 4], -1).reshape(2 * I, H)].reshape(2 * I, -1, 32),
                  (L.shared_sf.cpu().numpy().astype(int) - 127)[..., None]).reshape(2 * I, H)
    assert d2.max() > 7
    q4 = L.q4.cpu().numpy()
    x4 = np.ldexp(E2M1_TABLE[np.stack([q4 & 15, q4 >> 4], -1).reshape(T, H)].reshape(T, -1, 32), (L.sf4.cpu().numpy().astype(int) - 127)[..., None]).reshape(T, H)
    x8 = np.ldexp(E4M3_TABLE[L.x_q.cpu().numpy()].reshape(T, -1, 32), (L.x_sf.cpu().numpy().astype(int) - 127)[..., None]).reshape(T, H)
    for got, x in ((L.up4, x4), (L.up8, x8)):
        r = x @ wv.T
        assert (np.abs(got.double().cpu().numpy() - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -12.9 * (np.abs(x) @ np.abs(wv).T)).all()
    # the balance and its gradient
    lg, ids = L.logits.double().cpu().numpy(), L.ids.cpu().numpy()
    b = balance_ref(lg, ids, L.off.cpu().numpy())
    assert np.array_equal(L.counts.cpu().numpy(), b["counts"]) and np.array_equal(L.rows.cpu().numpy(), b["rows"])
    assert np.allclose(L.loss.cpu().numpy(), b["loss"], rtol=2.0 ** -17) and np.allclose(L.z.cpu().numpy(), b["z"], rtol=2.0 ** -17)
    g = gate_grad_ref(lg, ids, b["counts"], b["rows"], d_loss=L.d_loss.cpu().numpy(), d_z=L.d_z.cpu().numpy(), d_topk_w=L.d_w.cpu().numpy(),
                      offsets=L.off.cpu().numpy(), scale=1.5)
    got = L.d_logits.cpu().numpy()
    assert (got[180:] == 0).all() and np.isnan(g[180:]).all()
    # every addend of an element is below 1e-2 here, and the sum loses 2^-17 of them
    assert np.abs(got[:180] - g[:180]).max() < 1e-2 * 2.0 ** -17 * 8


def test_layer_side_stream_bound_and_poisoned(gpu):
    L, x = Layer(gpu), draw(gpu, 2)
    L.calls(x)
    torch.cuda.synchronize()
    want = L.results()
    side = torch.cuda.Stream()
    L.spoil()
    side.wait_stream(torch.cuda.current_stream())
    L.calls(x, stream=side)
    side.synchronize()
    assert same(L.results(), want)
    bound = L.calls(x, bind=True)
    for _ in range(3):
        L.spoil()
        for c in bound:
            c()
        torch.cuda.synchronize()
        assert same(L.results(), want)


def test_layers_side_by_side(gpu):
    """Two layers with buffers of their own, at once on two streams."""
    A, C = Layer(gpu, 1), Layer(gpu, 2)
    xa, xc = draw(gpu, 3), draw(gpu, 4)
    A.calls(xa)
    C.calls(xc)
    torch.cuda.synchronize()
    wa, wc = A.results(), C.results()
    A.spoil()
    C.spoil()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        A.calls(xa, stream=s)
        C.calls(xc, stream=t)
    torch.cuda.synchronize()
    assert same(A.results(), wa) and same(C.results(), wc)


def test_layer_graphs_that_share_workspaces(gpu):
    """Two graphs over the same buffers and workspaces, replayed in turn with eager calls between them, each against
    the eager result of its input."""
    L = Layer(gpu, 3)
    xs = [draw(gpu, 5), draw(gpu, 6)]
    want, graphs = [], []
    for x in xs:
        L.calls(x)
        torch.cuda.synchronize()
        want.append(L.results())
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.calls(x)
        graphs.append(g)
    for i in (0, 1, 0, 0, 1, 1, 0):
        L.spoil()
        if i:
            L.calls(xs[1 - i])
        graphs[i].replay()
        torch.cuda.synchronize()
        assert same(L.results(), want[i]), i
    for x in xs:  # new inputs in the captured buffer
        x.copy_(draw(gpu, 7))
    graphs[0].replay()
    torch.cuda.synchronize()
    got = L.results()
    L.spoil()
    L.calls(xs[0])
    torch.cuda.synchronize()
    assert same(got, L.results())


@pytest.mark.parametrize("shape", [(1, 512, 96, "e4m3"), (100, 1024, 200, "e2m1"), (300, 1056, 130, "e4m3"), (700, 512, 3000, "e2m1"),
                                   (4200, 640, 4100, "e2m1"), (4200, 640, 4100, "e4m3")])
def test_every_product_kernel_in_a_graph(gpu, shape):
    T_, K_, N_, fmt = shape
    print(shape, flush=True)
    s = B.make_mx_linear(T_, K_, N_, fmt)
    q = torch.empty(T_, K_ // 2 if fmt == "e2m1" else K_, dtype=torch.uint8, device=gpu)
    sf, x = torch.empty(T_, K_ // 32, dtype=torch.uint8, device=gpu), torch.randn(T_, K_, device=gpu)
    wq, wsf = torch.empty(N_, K_ // 2, dtype=torch.uint8, device=gpu), torch.empty(N_, K_ // 32, dtype=torch.uint8, device=gpu)
    B.mx_quant(B.make_mx_quant(N_, K_, "e2m1", F32), torch.randn(N_, K_, device=gpu), wq, wsf)
    w = B.mx_linear_prepare(s, wq, wsf)
    y, ws = torch.empty(T_, N_, dtype=BF16, device=gpu), u8(gpu, B.mx_linear_workspace_bytes(s))

    def go():
        B.mx_quant(B.make_mx_quant(T_, K_, fmt, F32), x, q, sf)
        B.mx_linear(s, q, sf, w, y, ws)

    go()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for i in range(4):
        x.copy_(torch.randn(T_, K_, generator=torch.Generator().manual_seed(i)))
        go()
        torch.cuda.synchronize()
        want = y.clone()
        y.fill_(7)
        ws.fill_(0x7F)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_tensors_elsewhere_are_refused(gpu):
    L = Layer(gpu)
    with pytest.raises(ValueError):
        B.mx_linear(L.lin4, L.q4, L.sf4, L.shared, L.up4, L.lws.cpu())
    with pytest.raises(ValueError):
        B.mx_quant(L.quant, L.y, L.q4[:-1], L.sf4)
    with pytest.raises(TypeError):
        B.mx_quant(L.quant, L.y.float(), L.q4, L.sf4)
    with pytest.raises(ValueError):
        B.balance(L.bal, L.logits, L.ids, L.bws, seq_offsets=L.off[:-1], counts=L.counts)
    with pytest.raises(TypeError):
        B.balance(L.bal, L.logits, L.ids.int(), L.bws, seq_offsets=L.off, counts=L.counts)
    with pytest.raises(B.MoeError):
        B.balance(L.bal, L.logits, L.ids, L.bws, counts=L.counts)  # three sequences without offsets
    with pytest.raises(B.MoeError):
        B.mx_linear(B.make_mx_linear(300, 1056, 130, "e4m3"), u8(gpu, 300, 1056), u8(gpu, 300, 33),
                    u8(gpu, B.mx_linear_weight_bytes(B.make_mx_linear(300, 1056, 130))), torch.empty(300, 130, dtype=BF16, device=gpu))
    torch.cuda.synchronize()


def test_rows_behind_four_gibibytes(gpu):
    """Rows whose offsets pass 32 bits have the results of the same rows at the start."""
    block = 4096

    def far(n, row, dtype, seed, make):
        """[n, row] whose blocks of rows are all the same."""
        t = torch.empty(n, row, dtype=dtype, device=gpu)
        t.view(-1, block, row)[:] = make(torch.Generator(gpu).manual_seed(seed), (block, row)).to(dtype)
        return t

    def alike(*ts):
        for t in ts:
            assert torch.equal(t[:block], t[-block:])

    normal = lambda g, s: torch.randn(s, generator=g, device=gpu)  # noqa: E731
    # 270336 x 16384: 8.9 GB of x, 4.4 GB of codes and 2.2
    n, K, N = 66 * block, 16384, 96
    print("quant", flush=True)
    x = far(n, K, BF16, 1, normal)
    for fmt, width in (("e4m3", K), ("e2m1", K // 2)):
        q, sf = torch.empty(n, width, dtype=torch.uint8, device=gpu), torch.empty(n, K // 32, dtype=torch.uint8, device=gpu)
        B.mx_quant(B.make_mx_quant(n, K, fmt), x, q, sf)
        alike(q, sf)
        print("product", fmt, flush=True)
        s = B.make_mx_linear(n, K, N, fmt)
        w = B.mx_linear_prepare(s, *quantised(gpu, N, K))
        y, ws = torch.empty(n, N, dtype=BF16, device=gpu), u8(gpu, B.mx_linear_workspace_bytes(s))
        B.mx_linear(s, q, sf, w, y, ws)
        alike(y)
        few = B.make_mx_linear(block, K, N, fmt)
        z = torch.empty(block, N, dtype=BF16, device=gpu)
        B.mx_linear(few, q[-block:], sf[-block:], w, z, u8(gpu, B.mx_linear_workspace_bytes(few)))
        assert (z.float() - y[:block].float()).abs().max() <= 2.0 ** -7 * y[:block].float().abs().max()  # other sums: a step or two
        del q, sf, y, ws
    print("product with wide rows of y", flush=True)
    s = B.make_mx_linear(n, 64, N, "e2m1", y_stride=9000)
    q, sf = far(n, 32, torch.uint8, 2, lambda g, sh: torch.randint(0, 256, sh, generator=g, device=gpu)), \
        torch.full((n, 2), 127, dtype=torch.uint8, device=gpu)
    y = torch.empty(n, 9000, dtype=BF16, device=gpu)
    B.mx_linear(s, q, sf, B.mx_linear_prepare(s, *quantised(gpu, N, 64)), y[:, :N], u8(gpu, B.mx_linear_workspace_bytes(s)))
    alike(y[:, :N])
    del x, y
    print("balance and gradient", flush=True)
    n, E, k = 1056 * block, 257, 3
    logits = far(n, E, F32, 3, normal)
    ids = torch.topk(logits[:block], k)[1].repeat(n // block, 1)
    s = B.make_balance(n, E, k, num_seqs=3)
    off = torch.tensor([0, block, n - block, n], device=gpu)
    out = {"counts": torch.empty(3, E, dtype=torch.int32, device=gpu), "rows": torch.empty(3, dtype=torch.int32, device=gpu),
           "share": torch.empty(3, E, device=gpu), "loss": torch.empty(3, device=gpu)}
    B.balance(s, logits, ids, u8(gpu, B.balance_workspace_bytes(s)), seq_offsets=off, **out)
    assert torch.equal(out["counts"][0], out["counts"][2]) and torch.equal(out["counts"][1], out["counts"][0] * (n // block - 2))
    assert out["rows"].tolist() == [block, n - 2 * block, block]
    for t in (out["share"], out["loss"]):  # sums of 2^22 values by lanes, waves and tiles
        assert (t - t[:1]).abs().max() <= 2.0 ** -14 * t.abs().max()
    d = torch.empty(n, E, device=gpu)
    one = torch.ones(3, device=gpu)
    B.gate_grad(s, logits, ids, d, seq_offsets=off, counts=out["counts"], rows=out["rows"], d_loss=one,
                d_topk_w=torch.ones(n, k, device=gpu))
    alike(d)
    torch.cuda.synchronize()


def quantised(dev, N, K):
    q, sf = torch.empty(N, K // 2, dtype=torch.uint8, device=dev), torch.empty(N, K // 32, dtype=torch.uint8, device=dev)
    B.mx_quant(B.make_mx_quant(N, K, "e2m1", F32), torch.randn(N, K, generator=torch.Generator(dev).manual_seed(N), device=dev), q, sf)
    return q, sf
