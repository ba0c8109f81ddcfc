"""The whole-layer decode against the bound that its documented roundings give (tests/_layer_bound.py): element by
element, in the mean, where x and h span more than fp16's range, and with scales that are no numbers."""
import numpy as np
import pytest
import torch

from tests import _layer_bound as lb
from tests import _layer_ref as ref
from tests.test_gpu_moe_decode import SHAPES, Layer, g, same_bits  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().double().numpy()


def compare(lay, in_the_mean=False):
    lay.call()
    out, ids, _, logits = lay.result()
    want_ids, p = ref.topk(logits.cpu().numpy(), lay.bias, lay.k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    want, bound = lb.layer(lay.fmt, ref.f64(lay.x), want_ids, p, lay.w1, lay.s1, lay.w2, lay.s2)
    err = np.abs(ref.f64(out) - want)
    assert np.all(err <= bound), f"worst error / bound {np.nanmax(err / bound):.3g}"
    if in_the_mean:
        r, limit = lb.rms(ref.f64(out), want), lb.rms_limit(lay.fmt, want, bf16)
        assert r <= limit, (r, limit)
    return want


@pytest.mark.parametrize("fmt,T,E,k,H,I", SHAPES)
def test_every_element(g, fmt, T, E, k, H, I):
    compare(Layer(g, fmt, T, E, k, H, I, seed=T * 17 + I))


@pytest.mark.parametrize("fmt,T,E,k,H,I", [("nf4", 8, 64, 8, 2048, 1024), ("mxfp4", 8, 16, 8, 2048, 512),
                                           ("mxfp4", 6, 12, 4, 2880, 2880), ("nf4", 8, 8, 2, 7168, 320)])
def test_the_mean_error_is_that_of_the_stated_roundings(g, fmt, T, E, k, H, I):
    compare(Layer(g, fmt, T, E, k, H, I, router=False, seed=501 + H), in_the_mean=True)


def zero_codes(lay, name, columns):
    """Sets the codes of the given k columns of a stack to zero (NF4 code 7, e2m1 code 0)."""
    w, z = getattr(lay, name), 7 if lay.fmt == "nf4" else 0
    for c in columns:
        high = (c % 2 == 0) == (lay.fmt == "nf4")  # NF4: the even element in the high nibble, MXFP4 in the low one
        b = w[:, :, c // 2]
        w[:, :, c // 2] = (b & 0x0F) | (z << 4) if high else (b & 0xF0) | z
    lay.d[name].copy_(torch.from_numpy(w))


@pytest.mark.parametrize("fmt", ["mxfp4", "nf4"])
@pytest.mark.parametrize("drop", [20, 30, 36, 44])
def test_small_values_of_x_beside_large_ones(g, fmt, drop):
    """The large half of x meets zero codes: the result comes from values 2^-drop of the largest alone."""
    lay = Layer(g, fmt, 3, 4, 2, 256, 128, router=False, seed=521)
    x = lay.x.float()
    x[:, 1::2] *= 2.0 ** -drop
    lay.x = x.bfloat16()
    lay.dx.copy_(lay.x)
    zero_codes(lay, "w1", range(0, 256, 2))
    lay.s1 = lay.s1 + np.uint8(min(drop, 100) // 2) if fmt == "mxfp4" else lay.s1 * np.float32(2.0 ** (drop // 2))
    lay.d["s1"].copy_(torch.from_numpy(lay.s1))
    want = compare(lay)
    assert np.abs(want).max() > 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nf4"])
@pytest.mark.parametrize("drop", [20, 30, 36, 44])
@pytest.mark.parametrize("T,E,k,H,I", [(3, 4, 2, 256, 128), (8, 16, 8, 128, 1024)])  # h in shared, in global memory
def test_small_values_of_h_beside_large_ones(g, fmt, drop, T, E, k, H, I):
    """Every other up row is 2^drop larger, and its h meets zero codes in the down projection."""
    lay = Layer(g, fmt, T, E, k, H, I, router=False, seed=541)
    s = lay.s1[:, I::2]
    s[...] = s + np.uint8(drop) if fmt == "mxfp4" else s * np.float32(2.0 ** drop)
    lay.d["s1"].copy_(torch.from_numpy(lay.s1))
    zero_codes(lay, "w2", range(0, I, 2))
    want = compare(lay)
    assert np.abs(want).max() > 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("stack", ["s1", "s2"])
def test_nf4_absmax_that_is_no_number_reaches_the_tokens_that_chose_the_expert(g, value, stack):
    lay = Layer(g, "nf4", 4, 6, 2, 256, 128, router=False, seed=561)
    lay.call()
    clean, ids = lay.result()[:2]
    e, row = int(ids[0, 0]), 37
    lay.d[stack][e, row, -1] = value
    lay.call()
    out = lay.result()[0]
    hit = (ids == e).any(dim=1)
    assert hit.any() and not hit.all()
    assert same_bits(out[~hit], clean[~hit])
    if stack == "s1":  # a gate row: its h is NaN, an infinity or, where silu is 0, NaN again or 0
        bad = ~torch.isfinite(out[hit])
        assert torch.all(bad.all(dim=1) | ~bad.any(dim=1))
        if value != value:
            assert bad.all()
    else:  # one output
        others = [c for c in range(256) if c != row]
        assert not torch.isfinite(out[hit][:, row]).any()
        assert same_bits(out[:, others], clean[:, others])
