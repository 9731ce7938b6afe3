"""GPU tests of the grouped linear operators at the values where an activation, its slope or the
checkpoint's codes can go wrong: exact zeros, far tails, steps of the quantisation."""
import math

import pytest
import torch

import linear_reference as R
import sparse_mixture_experts_26_b200 as moe

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- exact zeros under a ReLU
# shares of a long reduction, single SMs, pairs; one group; blocks that end inside 32 features
@pytest.mark.parametrize("counts,K,N", [((5, 0, 20), 128, 136), ((300, 260), 128, 264),
                                        ((1100, 900), 128, 264), ((6, 0, 3), 8192, 40),
                                        ((70,), 64, 8)])
def test_relu_gradient_of_exact_zeros(counts, K, N):
    """z are whole numbers, many of them zero beside live ones: the slope there is 0."""
    n, E = sum(counts), len(counts)
    g = torch.Generator(device="cuda").manual_seed(n + K)

    def whole(*shape, most=2):
        return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(bf)

    x, W, dy = whole(n, K), whole(E, N, K), whole(n, N, most=8)
    x[::7] = 0            # rows whose z is all zero
    W[:, ::3] = 0         # pruned features
    off = R.offsets_of(counts)
    ws = moe.alloc_grouped_linear_workspace(n, K, N, E)
    bws = moe.alloc_grouped_linear_backward_workspace(n, K, N, E)
    y = torch.empty(n, N, dtype=bf, device="cuda")
    codes, scales = moe.alloc_checkpoint(n, N)
    moe.moe_grouped_linear_train(x, off, W, y, codes, scales, ws, act="relu")
    z, _ = R.grouped_z(x, W, None, counts)
    assert bool((z == 0).any()) and bool((z != 0).any())
    kept = R.values(codes, scales)
    assert bool(((kept > 0) == (z > 0)).all())
    assert bool(((kept - z).abs() <= R.half_step(scales, N) * (1 + 2.0 ** -13)).all())
    dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty(E, N, device="cuda")
    moe.moe_grouped_linear_backward(dy, x, off, W, bws, dx=dx, dW=dW, db=db, codes=codes,
                                    scales=scales, act="relu")
    (rx, rW, rb), _ = R.gradients(dy, x, W, z, "relu", counts)
    # sums of whole numbers below 2^24: exact, up to the one rounding to bf16
    assert torch.equal(db.double(), rb)
    assert torch.equal(dx, rx.to(bf)) and torch.equal(dW, rW.to(bf))
    assert not bool(dW[:, ::3].any())
