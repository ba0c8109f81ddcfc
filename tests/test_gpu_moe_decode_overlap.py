"""Whole-layer decode calls beside other work: the launch needs every SM at once, so calls on two streams, two graphs,
two branches of one graph, and beside kernels of another stream take turns, and none waits for the other's end."""
import pytest
import torch

from tests.test_gpu_moe_decode import Layer, g, same_bits  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def layers(g, seed):
    lays = [Layer(g, f, T, 24, 6, 1024, 512, seed=seed + T) for f, T in (("nf4", 8), ("mxfp4", 5))]
    want = []
    for lay in lays:
        lay.call()
        want.append(lay.result())
        lay.out.fill_(9.0)
    torch.cuda.synchronize()
    return lays, want


def check(lays, want):
    for lay, w in zip(lays, want):
        for a, b in zip(lay.result(), w):
            assert same_bits(a, b)


def test_two_graphs_replayed_on_two_streams(g):
    lays, want = layers(g, 601)
    graphs = []
    for lay in lays:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _ in range(5):
                lay.call()
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in lays]
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    check(lays, want)


def test_two_branches_of_one_graph(g):
    lays, want = layers(g, 621)
    gr = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(gr):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for _ in range(5):
            lays[0].call()
            with torch.cuda.stream(side):
                lays[1].call()
        main.wait_stream(side)
    for _ in range(20):
        gr.replay()
    check(lays, want)


def test_beside_kernels_of_another_stream(g):
    lays, want = layers(g, 641)
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        with torch.cuda.stream(st):
            a = (a @ a).clamp_(-1, 1)
        for lay in lays:
            lay.call()
    check(lays, want)


def test_between_kernels_that_start_early(g):
    """Before and after calls that use programmatic launches: the decode waits for the first, the second for it."""
    lay = Layer(g, "mxfp4", 8, 16, 4, 512, 256, router=False, seed=661)
    M, I = 32, 256
    gu = torch.randn(M, 2 * I, device="cuda").bfloat16()
    h, codes, scales = (torch.empty(M, n, dtype=d, device="cuda") for n, d in
                        ((I, torch.bfloat16), (2 * I, torch.uint8), (2 * I // 32, torch.uint8)))
    lay.call()
    x0, first = lay.dx.clone(), lay.result()[0]
    ids = torch.arange(8, dtype=torch.int32, device="cuda")
    moved = torch.empty(8, 512, dtype=torch.bfloat16, device="cuda")
    for _ in range(20):
        lay.dx.zero_()
        # x is written by a gather that launches early, the output gathered on by another one
        g.combine_backward(x0, ids, None, lay.dx, k=1)
        lay.call()
        g.combine_backward(lay.out, ids, None, moved, k=1)
        g.swiglu_ckpt8(gu, h, codes, scales)
    torch.cuda.synchronize()
    assert same_bits(moved, first) and same_bits(lay.result()[0], first)
