"""The 8-bit SwiGLU checkpoint and its backward pass at the top of bf16's range."""
import numpy as np
import pytest
import torch

from tests import _layer_ref as ref
from tests.test_gpu_training_step import U, bf, g, run_forward  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

@pytest.mark.parametrize("x", [0.5, 1.0, 2.0, 4.0, 30.0])
def test_backward_where_slope_times_up_passes_fp32(g, x):
    """silu'(x) u dh is an ordinary number, silu'(x) u is not: silu' is at most 1.1, u 1.875 2^127."""
    M, I = 2, 32
    a = np.full((M, 2 * I), x)
    a[:, I:] = 1.875 * 2.0 ** 127
    dh = bf(np.full((M, I), 2.0 ** -10))
    _, codes, scales = run_forward(g, bf(a), I)
    dgu = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    g.swiglu_ckpt8_backward(dh.cuda(), codes, scales, dgu)
    torch.cuda.synchronize()
    s = ref.sigmoid(x)
    want = np.concatenate([2.0 ** -10 * a[:, I:] * s * (1 + x * (1 - s)), np.full((M, I), 2.0 ** -10 * x * s)], 1)
    assert np.all(np.abs(ref.f64(dgu) - want) <= (U + 2.0 ** -18) * np.abs(want))
