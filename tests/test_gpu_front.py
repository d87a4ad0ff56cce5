"""The calls in front of the experts run together as an MoE layer uses them: norm, router product, gate, the
forward, and the next norm; eager, on a side stream and as replays of one graph."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B
from moe_expert_ffn_plan_amd import inputs
from oracle.forward import forward_ref
from oracle.front import gate_ref, norm_ref, router_ref
from parity import assert_y_gate, fp8_values

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
T, H, I, E, K, GROUPS, KEPT = 96, 512, 256, 16, 4, 4, 2
W = inputs.Workload("front", T, H, I, E, E, K, 16, "uniform", seed=41, weight_seed=51)


class Layer:
    """Buffers and weights of one MoE layer on the GPU."""

    def __init__(self, dev, router_dtype=F32):
        g = torch.Generator().manual_seed(42)
        self.weights = inputs.make_weights(W, device="cpu")
        self.moe = B.shape_of(W)
        self.tiled = B.prepare_all(self.moe, {k: v.to(dev) for k, v in self.weights.items()})
        self.norm = B.make_norm(T, H, 1e-6)
        self.router = B.make_router(T, H, E, weight_dtype=router_dtype)
        self.gate = B.make_gate(T, E, K, score="sigmoid", num_groups=GROUPS, topk_groups=KEPT, group_score="top2",
                                scale=2.5)
        self.norm_w = (1 + 0.1 * torch.randn(H, generator=g)).to(BF16).to(dev)
        self.router_w = (torch.randn(E, H, generator=g) / H ** 0.5).to(router_dtype).to(dev)
        self.router_t = B.router_prepare(self.router, self.router_w)
        self.bias = torch.randint(-50, 51, (E,), generator=g).float().to(dev) * 1e-3
        def u8(*s):
            return torch.empty(*s, dtype=torch.uint8, device=dev)
        self.x_q, self.x_sf = u8(T, H), u8(T, H // 32)
        self.y = torch.empty(T, H, dtype=BF16, device=dev)
        self.logits = torch.empty(T, E, dtype=F32, device=dev)
        self.ids = torch.empty(T, K, dtype=torch.int64, device=dev)
        self.w = torch.empty(T, K, dtype=F32, device=dev)
        self.out = torch.empty(T, H, dtype=BF16, device=dev)
        self.ws = torch.full((B.forward_workspace_bytes(self.moe),), 0x5A, dtype=torch.uint8, device=dev)
        self.rws = torch.full((B.router_workspace_bytes(self.router),), 0x5A, dtype=torch.uint8, device=dev)

    def run(self, x, residual, stream=None):
        """One layer: residual is updated in place, the layer's output lands in self.out."""
        B.norm_quant(self.norm, x, self.norm_w, self.x_q, self.x_sf, self.y, residual, residual, stream=stream)
        B.router_logits(self.router, self.y, self.router_t, self.logits, self.rws, stream=stream)
        B.gate(self.gate, self.logits, self.ids, self.w, bias=self.bias, stream=stream)
        t = self.tiled
        B.forward(self.moe, self.x_q, self.x_sf, self.ids, self.w, t["w1"], t["w1_sf"], t["w2"], t["w2_sf"], self.out,
                  self.ws, stream=stream)


def draw(dev, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=g).to(BF16).to(dev), (3 * torch.randn(T, H, generator=g)).to(BF16).to(dev)


def state(layer, residual):
    return [t.clone() for t in (residual, layer.y, layer.x_q, layer.x_sf, layer.logits, layer.ids, layer.w, layer.out)]


def same(a, b):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("router_dtype", [BF16, F32])
def test_layer_against_the_oracle(gpu, router_dtype):
    """Each stage against the oracle on that stage's inputs, over two layers that share the residual."""
    L = Layer(gpu, router_dtype)
    x, residual = draw(gpu, 1)
    for _ in range(2):
        r0 = residual.clone()
        x0 = x.clone()
        L.run(x, residual)
        torch.cuda.synchronize()
        h, v, code, _ = norm_ref(f64(x0), f64(L.norm_w), 1e-6, f64(r0))
        assert (np.abs(f64(residual) - h) <= np.abs(h) * 2.0 ** -8 * (1 + 2.0 ** -12)).all()
        assert (np.abs(f64(L.y) - v) <= np.abs(v) * 2.0 ** -8 * (1 + 2.0 ** -12)).all()
        q, sf = L.x_q.cpu().numpy(), L.x_sf.cpu().numpy()
        assert np.array_equal(sf, code)
        # half a step of E4M3 at the block's scale
        step = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * np.repeat(np.ldexp(1.0, code.astype(int) - 127), 32, 1))
        assert (np.abs(fp8_values(q, sf) - v) <= step * (1 + 2.0 ** -16)).all()
        yd, wd = f64(L.y), f64(L.router_w)
        n = H * (3 if router_dtype == F32 else 1)
        assert (np.abs(f64(L.logits) - router_ref(yd, wd)) <= n * 2.0 ** -23 * router_ref(np.abs(yd), np.abs(wd))).all()
        ids, w = gate_ref(f64(L.logits), K, "sigmoid", f64(L.bias), GROUPS, KEPT, "top2", scale=2.5)
        assert np.array_equal(L.ids.cpu().numpy(), ids)
        assert (np.abs(f64(L.w) - w) <= 2.0 ** -23 * w).all()
        n = {k: t.numpy() for k, t in L.weights.items()}
        ref = forward_ref(q, sf, ids, L.w.cpu().numpy(), n["w1"], n["w1_sf"], n["w2"], n["w2_sf"], num_experts=E,
                          expert_begin=0, block_m=W.block_m)
        assert_y_gate(L.out.float().cpu().numpy(), ref["y"])
        x = L.out.clone()


def test_layer_on_a_side_stream(gpu):
    """Calls on a stream of their own, handed over explicitly and as the current one."""
    L = Layer(gpu)
    x, r = draw(gpu, 2)
    ref = r.clone()
    L.run(x, ref)
    torch.cuda.synchronize()
    want = state(L, ref)
    side = torch.cuda.Stream()
    for explicit in (True, False):
        mine = r.clone()
        side.wait_stream(torch.cuda.current_stream())
        if explicit:
            L.run(x, mine, stream=side)
        else:
            with torch.cuda.stream(side):
                L.run(x, mine)
        side.synchronize()
        assert same(state(L, mine), want)


def test_two_layers_at_once(gpu):
    """Two layers with buffers of their own, on two streams at the same time."""
    layers, data = [Layer(gpu), Layer(gpu, BF16)], [draw(gpu, 3), draw(gpu, 4)]
    want = []
    for L, (x, r) in zip(layers, data):
        ref = r.clone()
        L.run(x, ref)
        torch.cuda.synchronize()
        want.append(state(L, ref))
    # without the forward, whose single launch wants the GPU to itself
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        rs = [r.clone() for _, r in data]
        torch.cuda.synchronize()
        for L, (x, _), r, s in zip(layers, data, rs, streams):
            B.norm_quant(L.norm, x, L.norm_w, L.x_q, L.x_sf, L.y, r, r, stream=s)
            B.router_logits(L.router, L.y, L.router_t, L.logits, L.rws, stream=s)
            B.gate(L.gate, L.logits, L.ids, L.w, bias=L.bias, stream=s)
        torch.cuda.synchronize()
        for L, r, w in zip(layers, rs, want):
            assert same(state(L, r)[:7], w[:7])


def test_layer_graph_replays(gpu):
    """The whole layer recorded once and replayed on new inputs, eager work between the replays."""
    L = Layer(gpu)
    x, r = draw(gpu, 5)
    L.run(x, r)           # eager once before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run(x, r)
    torch.cuda.synchronize()
    other = Layer(gpu)
    for seed in (6, 7, 8, 6):
        nx, nr = draw(gpu, seed)
        x.copy_(nx)
        r.copy_(nr)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = state(L, r)
        other.run(nx, nr)
        torch.cuda.synchronize()
        assert same(got, state(other, nr))


def test_padding_rows_reach_no_expert(gpu):
    """Rows of -infinity logits get id -1, which the plan drops: their output is zero."""
    L = Layer(gpu)
    x, r = draw(gpu, 9)
    L.run(x, r)
    torch.cuda.synchronize()
    full = L.out.clone()
    L.logits[T // 2:] = float("-inf")
    B.gate(L.gate, L.logits, L.ids, L.w, bias=L.bias)
    t = L.tiled
    B.forward(L.moe, L.x_q, L.x_sf, L.ids, L.w, t["w1"], t["w1_sf"], t["w2"], t["w2_sf"], L.out, L.ws)
    torch.cuda.synchronize()
    assert (L.ids[T // 2:] == -1).all() and (L.out[T // 2:] == 0).all()
    assert torch.equal(L.out[:T // 2], full[:T // 2])


def test_bound_calls(gpu):
    """Calls marshalled once give what the plain calls give."""
    L = Layer(gpu)
    x, r = draw(gpu, 10)
    mine = r.clone()
    L.run(x, mine)
    torch.cuda.synchronize()
    want = state(L, mine)
    mine = r.clone()
    calls = [B.norm_quant(L.norm, x, L.norm_w, L.x_q, L.x_sf, L.y, mine, mine, bind=True),
             B.router_logits(L.router, L.y, L.router_t, L.logits, L.rws, bind=True),
             B.gate(L.gate, L.logits, L.ids, L.w, bias=L.bias, bind=True)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    assert same(state(L, mine)[:7], want[:7])


def test_weights_prepared_on_a_side_stream(gpu):
    """Prepared weights do not share memory with pending work of the current stream, which is still to write it."""
    L = Layer(gpu)
    want, moe = L.router_t.clone(), {k: v.to(gpu) for k, v in L.weights.items()}
    a = torch.randn(4096, 4096, device=gpu)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(60):                                    # keeps the current stream busy
        a = (a @ a).clamp_(-1, 1)
    for t in (L.router_t, *L.tiled.values()):
        torch.empty_like(t).fill_(7)                       # written after that, and free at once
    got = B.router_prepare(L.router, L.router_w, stream=side)
    tiled = B.prepare_all(L.moe, moe, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(torch.equal(tiled[k], L.tiled[k]) for k in tiled)


def poison(layer):
    """Every output buffer and workspace of the layer to values that no call leaves there (on the current stream)."""
    layer.x_q.fill_(0x55), layer.x_sf.fill_(0x55), layer.ws.fill_(0x5A), layer.rws.fill_(0x5A)
    for t in (layer.y, layer.logits, layer.w, layer.out):
        t.fill_(float("nan"))
    layer.ids.fill_(777)


@pytest.mark.parametrize("explicit", [True, False])
def test_layer_on_a_side_stream_from_nothing(gpu, explicit):
    """The stream writes every output itself: its buffers are poisoned on it, after a pause, before each run; a call that
    went to another stream would be overwritten, one that read too early would see the poison."""
    L = Layer(gpu)
    side = torch.cuda.Stream()
    pause = torch.randn(2048, 2048, device=gpu)
    for seed in (12, 13):
        x, r = draw(gpu, seed)
        ref = r.clone()
        L.run(x, ref)
        torch.cuda.synchronize()
        want, mine = state(L, ref), r.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                pause = (pause @ pause).clamp_(-1, 1)
            poison(L)
            if not explicit:
                L.run(x, mine)
        if explicit:
            L.run(x, mine, stream=side)
        side.synchronize()
        assert same(state(L, mine), want)


def test_two_layers_at_once_from_nothing(gpu):
    layers, data = [Layer(gpu), Layer(gpu, BF16)], [draw(gpu, 14), draw(gpu, 15)]
    want = []
    for L, (x, r) in zip(layers, data):
        ref = r.clone()
        L.run(x, ref)
        torch.cuda.synchronize()
        want.append(state(L, ref))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        rs = [r.clone() for _, r in data]
        for L in layers:
            poison(L)
        torch.cuda.synchronize()
        for L, (x, _), r, s in zip(layers, data, rs, streams):
            B.norm_quant(L.norm, x, L.norm_w, L.x_q, L.x_sf, L.y, r, r, stream=s)
            B.router_logits(L.router, L.y, L.router_t, L.logits, L.rws, stream=s)
            B.gate(L.gate, L.logits, L.ids, L.w, bias=L.bias, stream=s)
        torch.cuda.synchronize()
        for L, r, w in zip(layers, rs, want):
            assert same(state(L, r)[:7], w[:7])


def test_bound_calls_from_nothing(gpu):
    """Bound calls write every output, each time they are called, on the stream that they are given."""
    L = Layer(gpu)
    x, r = draw(gpu, 16)
    mine = r.clone()
    calls = [B.norm_quant(L.norm, x, L.norm_w, L.x_q, L.x_sf, L.y, mine, mine, bind=True),
             B.router_logits(L.router, L.y, L.router_t, L.logits, L.rws, bind=True),
             B.gate(L.gate, L.logits, L.ids, L.w, bias=L.bias, bind=True)]
    side = torch.cuda.Stream()
    for seed, stream in ((17, None), (18, side), (17, side)):
        nx, nr = draw(gpu, seed)
        ref = nr.clone()
        L.run(nx, ref)
        torch.cuda.synchronize()
        want = state(L, ref)
        x.copy_(nx), mine.copy_(nr)
        poison(L)
        torch.cuda.synchronize()
        for c in calls:
            c(stream)
        torch.cuda.synchronize()
        assert same(state(L, mine)[:7], want[:7])
