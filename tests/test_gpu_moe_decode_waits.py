"""The whole-layer decode's bounded waits: a meeting of the grid that cannot complete ends every CTA with an error
status, whatever copies it has in flight, and a zero-filled workspace makes the next call right again."""
import pytest
import torch

from tests.test_gpu_moe_decode import Layer, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture
def g():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from bit_grouped_moe_b200 import gnf4
    gnf4.device_errors(clear=True)
    yield gnf4
    assert gnf4.device_errors() == 0


# The workspace's first words are the parity and the arrivals at the three meetings of parity 0.  Arrivals that start
# at 2^32 - 1 wrap to 0 with the first CTA and end one short of the grid: every CTA's wait runs out (2^32 cycles, about
# 2 s).  Meeting 0 has no copies in flight, 1 and 2 (h too large for shared memory) have a ring of weights.
@pytest.mark.parametrize("fmt,meeting,T,E,k,H,I", [
    ("mxfp4", 0, 3, 8, 2, 256, 160), ("mxfp4", 1, 1, 8, 2, 2048, 1024), ("nf4", 1, 8, 64, 8, 1024, 768),
    ("mxfp4", 2, 8, 64, 8, 256, 1024), ("nf4", 2, 8, 64, 8, 2048, 768),
])
def test_a_meeting_that_cannot_complete_ends_with_an_error_status(g, fmt, meeting, T, E, k, H, I):
    lay = Layer(g, fmt, T, E, k, H, I, router=meeting == 0, seed=201 + meeting)
    lay.call()
    want = lay.result()
    lay.ws.zero_()
    lay.ws.view(torch.int32)[1 + meeting] = -1
    lay.out.fill_(7.0)
    lay.call()
    torch.cuda.synchronize()
    assert g.device_errors(clear=True) == g.DEVERR_TIMEOUT
    assert torch.all(lay.guard == 7.0)  # nothing was stored
    lay.ws.zero_()
    for _ in range(3):
        lay.call()
        for a, b in zip(lay.result(), want):
            assert same_bits(a, b)
    lay.check()
