"""moe_balance and moe_gate_grad where they can go wrong.  Tolerances as derived in test_gpu_balance.py."""
import numpy as np
import pytest
import torch

from test_gpu_balance import check_gradient, inputs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ---- more sequences than the lanes that the last rows fill

@pytest.mark.parametrize("behind", [0, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,S", [(1001, 64, 20), (1003, 33, 9), (9, 8, 30), (1, 8, 30), (1001, 128, 40), (7, 100, 200), (1001, 256, 50),
                                   (65, 384, 64), (101, 20, 101), (1025, 64, 1000), (9001, 16, 6000)])
def test_gradient_last_rows_of_many_sequences(gpu, T, E, S, score, behind):
    """Sequences of equal length, empty ones among them where there are more than rows; `behind`: rows that follow the last."""
    print(f"grad {T} x {E} in {S}", flush=True)
    end = max(T - behind, 0)
    off = torch.from_numpy(np.linspace(0, end, S + 1).round().astype(np.int64))
    l, ids, _ = inputs(T, E, 3, T + S, F32, 0.1)
    for seed in range(2):
        check_gradient(l, ids, off, gpu, score, True, 1.0, S, seed=seed)


# ---- renormalised weights that are formed again, over the largest of the chosen

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E,k", [(8, 1), (20, 3), (32, 9), (64, 2), (64, 11), (100, 3), (128, 20), (256, 8), (256, 40), (300, 6), (384, 33),
                                 (512, 5), (1000, 8), (1024, 64)])
def test_gradient_of_chosen_far_below_the_others(gpu, E, k, dtype, score):
    """As with a bias that outweighs the scores: the chosen experts' scores are below 2^-126 of the others'."""
    l, _, _ = inputs(33, E, k, E + k, dtype)
    g = torch.Generator().manual_seed(E)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(33)])
    low = -128.0 - torch.randint(0, 4, (33, k), generator=g).to(dtype)
    check_gradient(l.scatter(1, ids, low), ids, None, gpu, score, True, 1.0, 1, ("w",))
