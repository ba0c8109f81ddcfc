"""The 8-bit SwiGLU checkpoint at the top of bf16's range: every finite value stands for a finite value, and the
backward pass computes with it."""
import numpy as np
import pytest
import torch

from tests import _layer_ref as ref
from tests.test_gpu_training_step import U, bf, g, run_forward  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

TOP = 1.875 * 2.0 ** 127  # 240 2^120: the largest e4m3 multiple of 2^120 that fp32 holds


def values():
    """gate_up [8, 64]: the 128 bf16 values of the top binade with both signs, among smaller ones."""
    a = np.ones((8, 64))
    top = (1 + np.arange(128) / 128) * 2.0 ** 127
    a[:4, :32] = top.reshape(4, 32)
    a[:4, 32:] = 2.0 ** -60
    a[4:, :32] = 2.0
    a[4:, 32:] = -top.reshape(4, 32)
    a[1, 3], a[5, 40] = -a[1, 3], -a[5, 40]
    return a


def expected(a):
    q, sc = ref.ckpt8(a)
    return np.clip(q, -TOP, TOP), sc


def test_every_finite_value_is_stored_as_a_finite_one(g):
    a = values()
    h, codes, scales = run_forward(g, bf(a), 32)
    want, sc = expected(a)
    got = ref.decode_ckpt(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), sc) and np.array_equal(got, want)
    assert np.abs(got).max() == TOP and np.all(np.abs(got - a) <= 2.0 ** -4 * np.abs(a))
    hw = a[:, :32] * ref.sigmoid(a[:, :32]) * a[:, 32:]
    ok = np.abs(hw) < 2.0 ** 127
    assert ok[:4].all() and np.all(np.abs(ref.f64(h) - hw)[ok] <= (U + 2.0 ** -20) * np.abs(hw)[ok])


def test_an_infinity_beside_the_largest_values(g):
    a = values()
    a[0, 5], a[6, 50], a[7, 33] = np.inf, -np.inf, np.nan
    _, codes, scales = run_forward(g, bf(a), 32)
    want, sc = expected(a)
    got = ref.decode_ckpt(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), sc) and np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got).sum() == 3


def test_backward_of_the_largest_values(g):
    a = values()
    M, I = 8, 32
    dh = bf(np.ldexp(1 + np.arange(M * I).reshape(M, I) / 256.0, -10))
    _, codes, scales = run_forward(g, bf(a), I)
    out = [torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda"), torch.empty(M, I, dtype=torch.bfloat16, device="cuda")]
    dw = torch.empty(M, 1, device="cuda")
    idx = torch.arange(M, dtype=torch.int32, device="cuda")
    g.swiglu_ckpt8_backward(dh.cuda(), codes, scales, out[0], sorted_to_flat=idx, flat_to_sorted=idx, h=out[1], d_weights=dw)
    torch.cuda.synchronize()
    q = expected(a)[0]
    gt, u, d = q[:, :I], q[:, I:], ref.f64(dh)
    s = ref.sigmoid(gt)
    h = gt * s * u
    want = np.concatenate([d * u * s * (1 + gt * (1 - s)), d * gt * s], 1)
    got, gh = ref.f64(out[0]), ref.f64(out[1])
    # one bf16 rounding, and exp, division and a few fp32 operations; a saturated gate's slope and value are 0 in fp32
    # where the definition has e^-2^127
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= (U + 2.0 ** -18) * np.abs(want) + 2.0 ** -126)
    ok = np.abs(h) < 2.0 ** 127
    assert ok[:4].all() and np.all(np.abs(gh - h)[ok] <= (U + 2.0 ** -18) * np.abs(h)[ok] + 2.0 ** -126)
    dots, mag = (d * h).sum(1), np.abs(d * h).sum(1)
    assert np.all(np.abs(dw.cpu().numpy()[:, 0] - dots)[:4] <= (I * 2.0 ** -24 + 2.0 ** -18) * mag[:4])


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
