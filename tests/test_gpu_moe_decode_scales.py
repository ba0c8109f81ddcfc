"""The whole-layer decode with scale arrays at any address their header rule allows: MXFP4 scales at any byte, NF4
absmax at any multiple of 4, between bytes that are NaN as scales."""
import pytest
import torch

from tests.test_gpu_moe_decode import Layer, g, same_bits  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def moved(t, offset):
    """The same values `offset` bytes past a 256-byte boundary; the bytes around are 255 (a NaN as e8m0 or as fp32)."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    part = buf[256 + offset:256 + offset + n]
    part.copy_(t.reshape(-1).view(torch.uint8))
    return part, buf


@pytest.mark.parametrize("fmt,offset1,offset2", [("mxfp4", 1, 15), ("mxfp4", 7, 8), ("mxfp4", 12, 3), ("mxfp4", 16, 5),
                                                 ("nf4", 4, 12), ("nf4", 8, 4), ("nf4", 12, 8)])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 64, 64), (3, 3, 3, 192, 320), (8, 4, 2, 2048, 1088)])
def test_scales_at_any_offset(g, fmt, offset1, offset2, T, E, k, H, I):
    lay = Layer(g, fmt, T, E, k, H, I, router=False, seed=401 + H)
    lay.call()
    want = lay.result()
    keep = []
    for n, off in (("s1", offset1), ("s2", offset2)):
        lay.d[n], buf = moved(lay.d[n], off)
        assert lay.d[n].data_ptr() % 16 == off % 16
        keep.append((buf, buf.clone()))
    lay.out.fill_(7.0)
    lay.call()
    for a, b in zip(lay.result(), want):
        assert same_bits(a, b)
    for buf, was in keep:
        assert torch.equal(buf, was)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 32, 32), (2, 2, 1, 32, 96), (5, 3, 2, 96, 160)])
def test_the_shortest_rows_at_odd_offsets(g, T, E, k, H, I):
    """Rows of one to five scales: a 16-byte block holds several rows and, at the ends, bytes outside the array."""
    lay = Layer(g, "mxfp4", T, E, k, H, I, router=False, seed=431 + H)
    lay.call()
    want = lay.result()[0]
    for off in range(1, 16):
        s1, _a = moved(torch.from_numpy(lay.s1).cuda(), off)
        s2, _b = moved(torch.from_numpy(lay.s2).cuda(), 16 - off)
        lay.d["s1"], lay.d["s2"] = s1, s2
        lay.out.fill_(7.0)
        lay.call()
        assert same_bits(lay.result()[0], want), off
    lay.check()
