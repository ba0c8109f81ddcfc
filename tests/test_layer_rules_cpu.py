"""Refusals of the whole-layer and training calls, without a GPU: the shape rules of their header comments, the
arguments that need one another, host and misaligned pointers, short workspaces."""
import ctypes

import pytest
from hypothesis import given, settings, strategies as st

from bit_grouped_moe_b200 import build

SETTINGS = settings(max_examples=150, deadline=None, derandomize=True)
SHAPE, ARG, OK = 2, 1, 0
P16 = ctypes.c_void_p(16)  # aligned, not device memory; the host checks never read it


@pytest.fixture(scope="module")
def g():
    build.build()
    from bit_grouped_moe_b200 import gnf4
    return gnf4


def near(*bounds):
    return st.one_of(st.sampled_from(sorted({b + d for b in bounds for d in (-1, 0, 1)})),
                     st.integers(0, 1100).map(lambda n: 32 * n))


@SETTINGS
@given(T=st.integers(-2, 10), E=near(0, 1, 8, 1024), k=st.integers(-1, 40), H=near(0, 32, 64, 7168, 8192, 57344, 57376),
       I=near(0, 32, 64, 65536, 65568))
def test_moe_decode_rules(g, T, E, k, H, I):
    # "0 <= T <= 8, 1 <= E <= 1024, 1 <= k <= min(E, 32), H and I multiples of 64 (NF4) or 32 (MXFP4), H >= that,
    #  T*H <= 57344 and H <= 57344, that <= I <= 65536"
    for f, q in ((g._lib.gnf4_moe_decode_nf4, 64), (g._lib.gnf4_moe_decode_mxfp4, 32)):
        ok = (0 <= T <= 8 and 1 <= E <= 1024 and 1 <= k <= min(E, 32) and H >= q and H % q == 0 and H <= 57344
              and T * H <= 57344 and I >= q and I % q == 0 and I <= 65536)
        got = f(None, None, None, None, T, E, k, H, I, None, None, None, None, None, None, None, None, 0, None)
        assert got == ((OK if T == 0 else ARG) if ok else SHAPE), g.last_error()
        if ok and T > 0:
            assert "x is NULL" in g.last_error()


def test_moe_decode_workspace_bytes(g):
    f = g.moe_decode_workspace_bytes
    base = f(1, 1, 64, 128)
    assert base > 0 and base % 256 == 0
    assert f(8, 8, 7168, 2048) >= base + 64 * 2048 * 2
    assert f(2, 4, 2048, 1000) >= f(2, 4, 2048, 32)
    for bad in ((0, 1, 64, 64), (9, 1, 64, 64), (1, 0, 64, 64), (1, 33, 64, 64), (1, 1, 0, 64), (1, 1, 64, 0),
                (1, 1, 64, 65537), (1, 1, 57345, 64)):
        assert f(*bad) == 0, bad


@SETTINGS
@given(M=st.sampled_from([-5, -1, 0, 1, 7, 1 << 25, (1 << 31) - 1]), I=near(0, 32, 64, 65536, 1 << 20))
def test_ckpt8_rules(g, M, I):
    # "M >= 0, I >= 32 and I % 32 == 0, M*I <= 2^40"
    ok = M >= 0 and I >= 32 and I % 32 == 0 and M * I <= 1 << 40
    want = (OK if M == 0 else ARG) if ok else SHAPE
    assert g._lib.gnf4_swiglu_ckpt8(None, M, I, None, None, None, None, None) == want, g.last_error()
    assert g._lib.gnf4_swiglu_ckpt8_backward(None, None, None, None, None, None, None, M, I, None, None, None,
                                             None) == want, g.last_error()


def test_ckpt8_backward_arguments_that_need_one_another(g):
    f = g._lib.gnf4_swiglu_ckpt8_backward
    assert f(P16, P16, P16, None, None, None, P16, 4, 32, P16, None, None, None) == ARG  # weights, no sorted_to_flat
    assert "sorted_to_flat" in g.last_error()
    assert f(P16, P16, P16, None, None, P16, None, 4, 32, P16, None, P16, None) == ARG  # d_weights, no sorted_to_flat
    assert "sorted_to_flat" in g.last_error()
    assert f(P16, P16, P16, None, P16, None, None, 4, 32, P16, None, P16, None) == ARG  # d_weights, no flat_to_sorted
    assert "flat_to_sorted" in g.last_error()


@SETTINGS
@given(T=st.sampled_from([-1, 0, 1, 9, 1 << 20, 1 << 28, (1 << 31) - 1]), k=st.integers(-1, 9), N=st.one_of(near(0, 8), st.integers(-3, 40)))
def test_combine_backward_rules(g, T, k, N):
    # "T >= 0, k >= 1, T*k < 2^31, N >= 8 and N % 8 == 0"
    ok = T >= 0 and k >= 1 and T * k < 1 << 31 and N >= 8 and N % 8 == 0
    got = g._lib.gnf4_combine_backward(None, None, None, None, None, T, k, N, None, None, None)
    assert got == ((OK if T == 0 else ARG) if ok else SHAPE), g.last_error()


def test_combine_backward_d_weights_need_y(g):
    f = g._lib.gnf4_combine_backward
    assert f(P16, None, P16, P16, None, 2, 2, 8, P16, P16, None) == ARG and "y" in g.last_error()
    assert f(P16, P16, P16, None, None, 2, 2, 8, P16, P16, None) == ARG and "flat_to_sorted" in g.last_error()


@SETTINGS
@given(T=st.integers(-2, 3), E=near(0, 1, 32, 4096), k=st.integers(-1, 40))
def test_route_topk_backward_rules(g, T, E, k):
    # "T >= 0, 1 <= E <= 4096, 1 <= k <= min(E, 32)"
    ok = T >= 0 and 1 <= E <= 4096 and 1 <= k <= min(E, 32)
    got = g._lib.gnf4_route_topk_backward(None, None, None, T, k, E, None, None)
    assert got == ((OK if T == 0 else ARG) if ok else SHAPE), g.last_error()


def test_host_and_misaligned_pointers_are_refused(g):
    L = g._lib
    bad = ctypes.c_void_p(24)
    assert L.gnf4_swiglu_ckpt8(bad, 1, 32, None, P16, P16, P16, None) == ARG and "aligned" in g.last_error()
    assert L.gnf4_swiglu_ckpt8(P16, 1, 32, None, P16, P16, P16, None) == ARG and "device memory" in g.last_error()
    assert L.gnf4_combine_backward(P16, None, P16, None, None, 1, 1, 8, P16, None, None) == ARG
    assert "device memory" in g.last_error()
    assert L.gnf4_route_topk_backward(ctypes.c_void_p(2), P16, P16, 1, 1, 1, P16, None) == ARG
    assert "aligned" in g.last_error()
    args = [P16, None, None, P16, 1, 4, 2, 64, 64, P16, P16, P16, P16, P16, P16, P16, P16, 1 << 20, None]
    assert L.gnf4_moe_decode_nf4(*args) == ARG and "device memory" in g.last_error()


def test_refusals_are_counted(g):
    g.call_stats_get(None, reset=True)
    L = g._lib
    L.gnf4_moe_decode_mxfp4(None, None, None, None, 9, 4, 2, 64, 64, None, None, None, None, None, None, None, None, 0, None)
    L.gnf4_swiglu_ckpt8(None, 0, 32, None, None, None, None, None)
    assert g.call_stats_get("gnf4_moe_decode_mxfp4")["refused"] == 1
    s = g.call_stats_get("gnf4_swiglu_ckpt8")
    assert (s["calls"], s["refused"], s["engaged"]) == (1, 0, 0)
