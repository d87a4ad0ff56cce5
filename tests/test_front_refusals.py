"""Argument checks of the norm, router and gate calls: the C ABI's statuses and the binding's errors (no GPU)."""
import ctypes

import pytest
import torch

from moe_expert_ffn_plan_amd import binding as B

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)       # 8-byte aligned only


def norm(shape, x=FAKE, residual=None, weight=FAKE, residual_out=None, y=FAKE, x_q=FAKE, x_sf=FAKE):
    return B.lib().moe_norm_quant(ctypes.byref(shape), x, residual, weight, residual_out, y, x_q, x_sf, None)


NORM = dict(num_tokens=4, hidden=256)


@pytest.mark.parametrize("change,status", [
    (dict(num_tokens=-1), -2), (dict(num_tokens=1 << 28), -2), (dict(hidden=0), -2), (dict(hidden=-32), -2), (dict(hidden=(1 << 20) + 32), -2),
    (dict(hidden=48), -3), (dict(hidden=33), -3), (dict(eps=-1e-6), -2), (dict(eps=float("nan")), -2),
    (dict(eps=float("inf")), -2), (dict(x_stride=255), -2), (dict(x_stride=-256), -2), (dict(x_stride=260), -3),
    (dict(residual_stride=128), -2), (dict(residual_stride=257), -3), (dict(residual_out_stride=250), -2),
    (dict(residual_out_stride=258), -3), (dict(x_stride=1 << 41), -2)])
def test_norm_shapes(change, status):
    assert norm(B.make_norm(**{**NORM, **change})) == status


@pytest.mark.parametrize("field", ["x_type", "residual_type", "weight_type"])
def test_norm_types(field):
    for bad in (-1, 2):
        s = B.make_norm(**NORM)
        setattr(s, field, bad)
        assert norm(s) == -2


def test_norm_pointers():
    s = B.make_norm(**NORM)
    assert B.lib().moe_norm_quant(None, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, None) == -1
    assert norm(s, x=None) == -1 and norm(s, weight=None) == -1
    assert norm(s, y=None, x_q=None, x_sf=None) == -1           # nothing to write
    assert norm(s, x_q=None) == -1 and norm(s, x_sf=None) == -1  # one without the other
    for name in ("x", "residual", "weight", "residual_out", "y", "x_q"):
        assert norm(s, **{name: ODD}) == -3, name
    assert norm(B.make_norm(0, 256), x=None, weight=None, y=None, x_q=None, x_sf=None) == 0


def router(shape, x=FAKE, w=FAKE, logits=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return B.lib().moe_router_logits(ctypes.byref(shape), x, w, logits, ws, ws_bytes, None)


ROUTER = dict(num_tokens=4, hidden=256, num_experts=8)


@pytest.mark.parametrize("change,status", [
    (dict(num_tokens=-1), -2), (dict(num_tokens=1 << 28), -2), (dict(hidden=0), -2), (dict(hidden=100), -3), (dict(hidden=(1 << 20) + 32), -2),
    (dict(num_experts=0), -2), (dict(num_experts=1025), -2), (dict(x_stride=200), -2), (dict(x_stride=257), -3)])
def test_router_shapes(change, status):
    s = B.make_router(**{**ROUTER, **change})
    assert router(s) == status
    v = ctypes.c_size_t()
    assert B.lib().moe_router_weight_bytes(ctypes.byref(s), ctypes.byref(v)) == status
    assert B.lib().moe_router_workspace_bytes(ctypes.byref(s), ctypes.byref(v)) == status
    assert B.lib().moe_router_prepare(ctypes.byref(s), FAKE, FAKE, None) == status


def test_router_pointers():
    s = B.make_router(**ROUTER)
    lib = B.lib()
    assert lib.moe_router_logits(None, FAKE, FAKE, FAKE, FAKE, 0, None) == -1
    assert lib.moe_router_weight_bytes(ctypes.byref(s), None) == -1
    assert lib.moe_router_workspace_bytes(ctypes.byref(s), None) == -1
    assert lib.moe_router_prepare(ctypes.byref(s), None, FAKE, None) == -1
    assert lib.moe_router_prepare(ctypes.byref(s), FAKE, None, None) == -1
    assert lib.moe_router_prepare(ctypes.byref(s), ODD, FAKE, None) == -3
    for name in ("x", "w", "logits"):
        assert router(s, **{name: None}) == -1 and router(s, **{name: ODD}) == -3, name
    bad = B.make_router(**ROUTER)
    bad.weight_type = 2
    assert router(bad) == -2
    assert router(B.make_router(0, 256, 8), x=None, w=None, logits=None, ws=None, ws_bytes=0) == 0


@pytest.mark.parametrize("weight", [torch.bfloat16, torch.float32])
def test_router_workspace_sizes(weight):
    """Whole copies of the logits, 256 MB of them at most, over all of the allowed sizes."""
    for T in (0, 1, 16, 17, 129, 1024, 1025, 40000, 1 << 20, (1 << 28) - 1):
        for hidden in (32, 96, 2048, 7168, 1 << 20):
            for E in (1, 63, 64, 65, 257, 384, 385, 1024):
                need = B.router_workspace_bytes(B.make_router(T, hidden, E, weight_dtype=weight))
                assert need <= 1 << 28 and need % max(1, 4 * T * E) == 0 and need != 4 * T * E or need == 0


def test_router_workspace():
    """Every shape that needs a workspace refuses one that is missing, misaligned or a byte short."""
    seen = 0
    for T in (1, 64, 128, 1000, 4096, 65536):
        for weight in (torch.bfloat16, torch.float32):
            s = B.make_router(T, 7168, 256, weight_dtype=weight)
            need = B.router_workspace_bytes(s)
            if need == 0:
                continue
            seen += 1
            assert router(s, ws=None) == -1
            assert router(s, ws=ODD) == -3
            assert router(s, ws_bytes=need - 1) == -4
    print(f"{seen} shapes with a workspace")


def test_router_weight_bytes():
    assert B.router_weight_bytes(B.make_router(1, 64, 8)) == 16 * 64 * 2
    assert B.router_weight_bytes(B.make_router(1, 64, 17, weight_dtype=torch.float32)) == 32 * 64 * 6


def gate(shape, logits=FAKE, bias=None, ids=FAKE, w=FAKE):
    return B.lib().moe_gate(ctypes.byref(shape), logits, bias, ids, w, None)


GATE = dict(num_tokens=4, num_experts=32, topk=4)


@pytest.mark.parametrize("change", [
    dict(num_tokens=-1), dict(num_tokens=1 << 28, topk=1), dict(num_experts=0), dict(num_experts=1025), dict(topk=0), dict(topk=33),
    dict(num_experts=128, topk=65), dict(num_groups=0), dict(num_groups=5), dict(num_groups=128, num_experts=1024),
    dict(num_groups=4, topk_groups=0), dict(num_groups=4, topk_groups=5), dict(num_groups=16, topk_groups=1),
    dict(num_tokens=(1 << 28) - 1, topk=5), dict(scale=float("nan")), dict(scale=float("inf")), dict(logits_stride=31),
    dict(logits_stride=-32)])
def test_gate_shapes(change):
    assert gate(B.make_gate(**{**GATE, **change})) == -2


@pytest.mark.parametrize("field", ["score", "group_score", "renormalize", "logits_type"])
def test_gate_switches(field):
    for bad in (-1, 2):
        s = B.make_gate(**GATE)
        setattr(s, field, bad)
        assert gate(s) == -2


def test_gate_pointers():
    s = B.make_gate(**GATE)
    assert B.lib().moe_gate(None, FAKE, None, FAKE, FAKE, None) == -1
    assert gate(s, logits=None) == -1 and gate(s, ids=None) == -1 and gate(s, w=None) == -1
    at = lambda a: ctypes.c_void_p(a)  # noqa: E731
    assert gate(s, logits=at(0x10002)) == -3 and gate(s, bias=at(0x10002)) == -3
    assert gate(s, ids=at(0x10004)) == -3 and gate(s, w=at(0x10002)) == -3
    assert gate(B.make_gate(**GATE, logits_dtype=torch.bfloat16), logits=at(0x10001)) == -3
    assert gate(B.make_gate(0, 32, 4), logits=None, ids=None, w=None) == 0


def test_binding_refuses_other_tensors():
    """Types, shapes, strides and devices are checked before the library is called."""
    cpu = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.norm_quant(B.make_norm(4, 256), cpu, w, y=cpu)
    with pytest.raises(ValueError):
        B.router_logits(B.make_router(4, 256, 8), cpu, w, w)
    with pytest.raises(ValueError):
        B.gate(B.make_gate(4, 32, 4), torch.zeros(4, 32), torch.zeros(4, 4), torch.zeros(4, 4))
    with pytest.raises(TypeError):
        B.gate(B.make_gate(4, 32, 4), None, None, None)
    for bad in (lambda: B.make_norm(4, 256, x_dtype=torch.float16), lambda: B.make_router(4, 256, 8, torch.float16),
                lambda: B.make_gate(4, 32, 4, score="relu"), lambda: B.make_gate(4, 32, 4, group_score="sum")):
        with pytest.raises(KeyError):
            bad()


def test_binding_row_checks(monkeypatch):
    """Row shapes, strides and types, on tensors that only say they lie on a device."""
    class Said(torch.Tensor):
        is_cuda = True

    dev = torch.device("cpu")
    t = torch.zeros(4, 40).as_subclass(Said)
    assert B._rows(t, torch.float32, "x", dev, 4, 40, 0) is not None
    assert B._rows(t[:, :32], torch.float32, "x", dev, 4, 32, 40) is not None
    assert B._rows(None, torch.float32, "x", dev, 4, 40, 0) is None
    for args in ((torch.float32, "x", dev, 4, 32, 0), (torch.float32, "x", dev, 4, 40, 48)):
        with pytest.raises(ValueError):
            B._rows(t, *args)
    with pytest.raises(ValueError):
        B._rows(t[:, :32], torch.float32, "x", dev, 4, 32, 0)
    with pytest.raises(ValueError):
        B._rows(t.t(), torch.float32, "x", dev, 40, 4, 0)
    with pytest.raises(TypeError):
        B._rows(t, torch.bfloat16, "x", dev, 4, 40, 0)


def test_every_finite_eps_and_scale():
    """The largest finite values are allowed, either sign of the scale; no tokens, so that no GPU is asked for."""
    for v in (0.0, 1e-45, 3.1e38, torch.finfo(torch.float32).max):
        assert norm(B.make_norm(0, 256, eps=v)) == 0
        assert gate(B.make_gate(0, 32, 4, scale=v)) == 0 and gate(B.make_gate(0, 32, 4, scale=-v)) == 0


@pytest.mark.parametrize("weight", [torch.bfloat16, torch.float32])
def test_router_tiles_of_all_sizes(weight):
    """Tiles of 16 tokens have a grid axis of 65535 for them: no allowed size past 1024 tokens takes them, and the
    tiles of a launch times its threads fit 32 bits."""
    with pytest.raises(B.MoeError):
        B.router_tile(B.make_router(4, 48, 8))
    assert B.router_tile(B.make_router(0, 64, 8))[2] == 1
    rows = (1, 16, 1024, 1025, 1 << 17, 1 << 24, (1 << 24) + 1, (1 << 27) - 1, (1 << 27) + 1, 180_000_000, (1 << 28) - 1)
    for T in rows:
        for hidden in (32, 96, 7168, 1 << 20):
            for E in (1, 17, 64, 65, 129, 256, 257, 385, 513, 770, 1024):
                m, n, splits = B.router_tile(B.make_router(T, hidden, E, weight_dtype=weight))
                assert (m == 16) <= (T <= 1024), (T, hidden, E, m, n)
                tiles = -(-min(T, 1 << 24) // m) * -(-E // n) * splits
                assert tiles * (1024 if m == 16 else 512) < 1 << 32, (T, hidden, E, m, n)


@pytest.mark.parametrize("weight", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hidden,E", [(7168, 256), (7168, 384), (4096, 64), (1 << 20, 1024), (512, 40), (64, 8), (32, 300)])
def test_router_workspace_of_the_most_tokens(hidden, E, weight):
    """One workspace for all batches up to the largest, which may itself need none."""
    need = {T: B.router_workspace_bytes(B.make_router(T, hidden, E, weight_dtype=weight))
            for T in [*range(0, 700), *range(700, 40000, 131), 65536, 1 << 20, (1 << 24) + 1, (1 << 28) - 1]}
    before = seen = 0
    for T in sorted(need):
        seen = max(seen, need[T])
        most = B.router_max_workspace_bytes(B.make_router(T, hidden, E, weight_dtype=weight))
        assert max(seen, before) <= most <= 1 << 28, T
        before = most
    some = max(need, key=need.get)
    if need[some]:
        s = B.make_router(some, hidden, E, weight_dtype=weight)
        assert router(s, ws_bytes=need[some] - 1) == -4
    bad = B.make_router(4, 48, 8)
    assert B.lib().moe_router_max_workspace_bytes(ctypes.byref(bad), ctypes.byref(ctypes.c_size_t())) == -3
    assert B.lib().moe_router_max_workspace_bytes(ctypes.byref(bad), None) == -1


def test_norm_in_place_needs_one_layout():
    """residual_out on the memory of x or the residual, but with rows elsewhere: one row's output on another's input."""
    at = lambda i: ctypes.c_void_p(0x10000 * i)  # noqa: E731
    for change in (dict(residual_stride=512), dict(residual_out_stride=264)):
        assert norm(B.make_norm(**NORM, **change), residual=at(2), residual_out=at(2)) == -2
    for change in (dict(x_stride=512), dict(residual_out_stride=264), dict(x_dtype=torch.float32),
                   dict(x_dtype=torch.float32, x_stride=264, residual_out_stride=264)):
        assert norm(B.make_norm(**NORM, **change), residual=at(2), residual_out=FAKE) == -2
        assert norm(B.make_norm(**NORM, **change), residual_out=FAKE) == -2
    # x and the residual are one buffer of two layouts: residual_out has to be that of both
    s = B.make_norm(**NORM, x_stride=512, residual_stride=256, residual_out_stride=256)
    assert norm(s, residual=FAKE, residual_out=FAKE) == -2


def test_prepared_weights_belong_to_the_stream(monkeypatch):
    """The tensors that router_prepare and prepare_weights return are allocated on the stream that writes them: on
    another, memory that its pending work still uses could be handed out."""
    class Said(torch.Tensor):
        is_cuda = True

    class Stream:
        cuda_stream = 7
        inside = False

        def __enter__(self):
            Stream.inside = True

        def __exit__(self, *_):
            Stream.inside = False

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    made, empty = [], torch.empty

    def recorded(*a, **kw):
        made.append(Stream.inside)
        return empty(*a, **kw).as_subclass(Said)

    monkeypatch.setattr(B, "lib", Lib)
    monkeypatch.setattr(B, "_here", lambda t, name: t.device)
    monkeypatch.setattr(B, "router_weight_bytes", lambda s: 1024)
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    w = torch.zeros(16, 32, dtype=torch.bfloat16).as_subclass(Said)
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8).as_subclass(Said)  # noqa: E731
    B.router_prepare(B.make_router(1, 32, 16), w, stream=Stream())
    B.prepare_weights(B.make_shape(1, 256, 256, 1, 1, 16), 1, u8(512 * 128), u8(512 * 8), stream=Stream())
    assert made == [True, True, True]


def test_gate_kernels_of_all_shapes():
    """Every kernel that any allowed shape takes is one that the GPU tests run by name."""
    from test_gpu_gate import KERNELS
    taken = set()
    for E in range(1, 1025):
        for groups in (d for d in range(1, 65) if E % d == 0):
            for k in (1, 8, 9, 16, 17, 64):
                if k <= E:
                    taken.add(B.gate_lanes(B.make_gate(1, E, k, num_groups=groups, topk_groups=groups)))
    assert taken == set(KERNELS)
    for kernel, shapes in KERNELS.items():
        for E, groups, kept, k in shapes:
            assert B.gate_lanes(B.make_gate(1, E, k, num_groups=groups, topk_groups=kept)) == kernel
    with pytest.raises(B.MoeError):
        B.gate_lanes(B.make_gate(1, 8, 9))
