"""moe_balance and moe_gate_grad where they can go wrong.  Tolerances as derived in test_gpu_balance.py."""
import numpy as np
import pytest
import torch

from test_gpu_balance import check_gradient, inputs

pytestmark = pytest.mark.gpu

F32 = torch.float32


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
