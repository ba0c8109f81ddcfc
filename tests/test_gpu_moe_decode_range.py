"""The whole-layer decode over fp32's range: sums and scales are fp32, so a result that fp32 holds comes out whatever
power of two its activations and its scales have."""
import numpy as np
import pytest
import torch

from bit_grouped_moe_b200 import inputs
from tests import _layer_ref as ref
from tests.test_gpu_moe_decode import Layer, g  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

SMALL, GLOBAL_H = (2, 3, 2, 128, 96), (8, 16, 8, 128, 1024)  # the second one's h is too large for shared memory


def scaled(g, fmt, shape, x_exp, e1, e2, seed):
    """Activations of 2^x_exp, scales of about 2^e1 (gate_up) and 2^e2 (down)."""
    T, E, k, H, I = shape
    if fmt == "nf4":
        H, I = -(-H // 64) * 64, -(-I // 64) * 64
    lay = Layer(g, fmt, T, E, k, H, I, router=False, seed=seed)
    rng = inputs.rng(seed + 50)
    for n, e in (("s1", e1), ("s2", e2)):
        old = getattr(lay, n)
        if fmt == "mxfp4":
            new = rng.integers(127 + e - 1, 127 + e + 2, size=old.shape, dtype=np.uint8)
        else:
            new = np.ldexp(rng.uniform(0.5, 1.5, size=old.shape), e).astype(np.float32)
        setattr(lay, n, new)
        lay.d[n].copy_(torch.from_numpy(new))
    lay.x = torch.ldexp(lay.x.float(), torch.tensor(x_exp)).bfloat16()
    lay.dx.copy_(lay.x)
    return lay


@pytest.mark.parametrize("shape", [SMALL, GLOBAL_H])
@pytest.mark.parametrize("fmt", ["mxfp4", "nf4"])
@pytest.mark.parametrize("x_exp,e1,e2", [
    (0, -24, 110),      # h near 2^-40, out near 2^74
    (0, -38, 120),      # h near 2^-68, out near 2^56
    (-60, 110, -110),   # gate_up near 2^54, h near 2^108, out near 1
    (-60, 56, 0),       # ordinary results of small activations
    (-90, 88, 0), (-120, 118, 0),
    (60, -62, 0), (90, -92, 50), (110, -112, -100),
    (0, -3, 112),       # down sums up to 2^118 of ordinary h
])
def test_results_that_fp32_holds(g, fmt, shape, x_exp, e1, e2):
    lay = scaled(g, fmt, shape, x_exp, e1, e2, seed=300 + abs(x_exp) + abs(e2))
    lay.call()
    lay.check()


@pytest.mark.parametrize("fmt", ["mxfp4", "nf4"])
@pytest.mark.parametrize("e1,e2", [(60, -60), (10, -5)])
def test_tokens_of_very_different_size_keep_their_own_range(g, fmt, e1, e2):
    """Tokens of 2^40, 1, 2^-40 and 2^-80, and router weights down to e^-60: the row of a token whose h fp32 holds is
    right, together with the others and alone, and that of one whose h passes fp32's range is not finite.

    Largest h with (60, -60): 2^214 and 2^133 of the first two tokens (MXFP4), 2^208 and 2^127.8 (NF4: too near the
    limit for a claim); with (10, -5) 2^114 at most."""
    T, E, k, H, I = 4, 8, 4, 128, 128
    lay = scaled(g, fmt, (T, E, k, H, I), 0, e1, e2, seed=351)
    lay.x = (lay.x.float() * torch.tensor([40.0, 0.0, -40.0, -80.0]).exp2()[:, None]).bfloat16()
    lay.dx.copy_(lay.x)
    lay.logits_in[:, :] = 0.0
    lay.logits_in[:, :4] = [30.0, 10.0, -10.0, -30.0]
    lay.logits_in[:, 4:] = -31.0
    lay.logits.copy_(torch.from_numpy(lay.logits_in))
    lay.call()
    out, ids, _, _ = lay.result()
    want_ids, p = ref.topk(lay.logits_in, None, k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    want, bound = ref.layer(fmt, ref.f64(lay.x), want_ids, p, lay.w1, lay.s1, lay.w2, lay.s2)
    top = np.zeros(T)  # largest |h| of a token over the experts it chose
    for t in range(T):
        for e in want_ids[t]:
            gu = ref.dequant(fmt, lay.w1[e], lay.s1[e]) @ ref.f64(lay.x)[t]
            top[t] = max(top[t], np.abs(gu[:I] * ref.sigmoid(gu[:I]) * gu[I:]).max())
    held = top < 2.0 ** 127
    assert held.sum() == (2 if e1 == 60 else T)
    assert np.all((np.abs(ref.f64(out) - want) <= bound)[held])
    assert not np.isfinite(ref.f64(out)[top > 2.0 ** 129]).any()
    for t in np.flatnonzero(held):
        one = torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
        f = g.moe_decode_nf4 if fmt == "nf4" else g.moe_decode_mxfp4
        f(lay.dx[t:t + 1], lay.d["w1"], lay.d["s1"], lay.d["w2"], lay.d["s2"], lay.logits[t:t + 1], lay.ids[:1].clone(),
          lay.p[:1].clone(), one, lay.new_workspace())
        torch.cuda.synchronize()
        assert np.all(np.abs(ref.f64(one[0]) - want[t]) <= bound[t])
