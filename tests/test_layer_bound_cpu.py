"""The decode's rms limit tells the stated roundings from coarser ones: a p * h of 11 bits stays below it, one of 8 bits
(bf16) does not, in either format; nor do NF4 codes of 8 bits."""
import numpy as np
import pytest
import torch

from bit_grouped_moe_b200 import inputs
from tests import _layer_bound as lb
from tests import _layer_ref as ref

T, E, k, H, I = 4, 3, 2, 4096, 128


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().double().numpy()


def f16(a):
    return (a / np.abs(a).max()).astype(np.float16).astype(np.float64) * np.abs(a).max()


@pytest.fixture(scope="module", params=["mxfp4", "nf4"])
def case(request):
    rng = inputs.rng(7)
    fmt = request.param
    if fmt == "nf4":
        w1, w2 = (rng.integers(0, 256, size=s, dtype=np.uint8) for s in ((E, 2 * I, H // 2), (E, H, I // 2)))
        s1, s2 = ((0.05 * rng.uniform(0.3, 1.5, size=s)).astype(np.float32) for s in ((E, 2 * I, H // 64), (E, H, I // 64)))
    else:
        (w1, s1), (w2, s2) = (inputs.mxfp4_random(rng, E, *s, e_lo=118, e_hi=122) for s in ((2 * I, H), (H, I)))
    x = bf16(rng.standard_normal((T, H)))
    ids, p = ref.topk(rng.standard_normal((T, E)).astype(np.float32), None, k)
    return fmt, (x, ids, p, w1, s1, w2, s2)


def test_eleven_bits_pass_and_eight_do_not(case):
    fmt, a = case
    want, bound = lb.layer(fmt, *a)
    limit = lb.rms_limit(fmt, want, bf16)
    fine = bf16(lb.layer(fmt, *a, round_h=f16)[0])
    assert lb.rms(fine, want) <= limit and np.all(np.abs(fine - want) <= bound)
    coarse = bf16(lb.layer(fmt, *a, round_h=bf16)[0])
    assert lb.rms(coarse, want) > 1.1 * limit


def test_codes_of_eight_bits_do_not_pass(case, monkeypatch):
    fmt, a = case
    if fmt != "nf4":
        return  # e2m1 is exact in bf16
    want, _ = lb.layer(fmt, *a)
    limit = lb.rms_limit(fmt, want, bf16)
    monkeypatch.setattr(ref, "NF4", bf16(ref.NF4))
    assert lb.rms(bf16(lb.layer(fmt, *a, round_h=f16)[0]), want) > 1.1 * limit
