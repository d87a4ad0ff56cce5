"""What the dense product says of its sizes (no GPU)."""
import pytest

from moe_expert_ffn_plan_amd import binding as B


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("K,N", [(512, 129), (1024, 384), (2048, 256), (4096, 384), (4096, 129), (7168, 640), (4064, 384), (7168, 2048)])
def test_largest_workspace_serves_every_smaller_batch(K, N, fmt):
    """Large batches go back and forth between kernels that have the scales laid out and kernels that do not."""
    sizes = sorted({*range(65, 300000, 1009), *range(32700, 32900, 16), 65526, 65587})
    need = 0
    for T in sizes:
        s = B.make_mx_linear(T, K, N, fmt)
        need = max(need, B.mx_linear_workspace_bytes(s))
        if T > 30000 and T % 7 == 0 or T in (65526, 65587, sizes[-1]):
            assert B.mx_linear_max_workspace_bytes(s) >= need, T


def test_largest_workspace_of_small_batches_is_that_of_one():
    for K, N in ((4096, 384), (4064, 1537)):
        for most in (0, 64, 130, 2000):
            need = max(B.mx_linear_workspace_bytes(B.make_mx_linear(T, K, N)) for T in range(most + 1))
            assert B.mx_linear_max_workspace_bytes(B.make_mx_linear(most, K, N)) == need


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_splits_are_those_that_run(fmt):
    """Every split has K-steps: ceil(steps / ceil(steps / splits)) of them is the number itself, and the workspace holds
    that many partial sums."""
    split = set()
    for steps in range(1, 80):
        for T, N in ((129, 64), (200, 512), (500, 1024), (1000, 1500)):
            s = B.make_mx_linear(T, 128 * steps, N, fmt)
            splits = B.mx_linear_tile(s)[2]
            per = -(-steps // splits)
            assert -(-steps // per) == splits, (steps, T, N)
            if splits > 1:
                assert B.mx_linear_workspace_bytes(s) == splits * T * -(-N // 64) * 64 * 4
                split.add(splits)
    assert len(split) > 3
