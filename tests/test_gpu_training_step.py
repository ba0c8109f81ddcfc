"""The training calls around the expert GEMMs: the 8-bit SwiGLU checkpoint, its backward pass, the backward of the
combine and of the router, each against its 64-bit definition, and a whole step of a routed layer against the
formula's gradients and against differences."""
import numpy as np
import pytest
import torch

from bit_grouped_moe_b200 import inputs
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -8  # half a step of bf16


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from bit_grouped_moe_b200 import gnf4
    gnf4.device_errors(clear=True)
    yield gnf4
    assert gnf4.device_errors() == 0


def bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16()


def same(a, b):
    v = lambda t: t.contiguous().view(torch.int16).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
    return bool(np.array_equal(v(a), v(b), equal_nan=t_float(a)))


def t_float(t):
    return t.dtype in (torch.float32, torch.float64)


def routing(rng, T, k, drop):
    """sorted_to_flat, flat_to_sorted, live rows: a random assignment of the live pairs to the first rows."""
    M = T * k
    live = np.sort(rng.permutation(M)[:M - int(round(M * drop))])
    s2f, f2s = np.full(M, -1, np.int32), np.full(M, -1, np.int32)
    s2f[:len(live)] = rng.permutation(live)
    f2s[s2f[:len(live)]] = np.arange(len(live), dtype=np.int32)
    return s2f, f2s, len(live)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------------------------------------ forward


def run_forward(g, gu, I, num_rows=None):
    M = gu.shape[0]
    h = torch.full((M, I), 7.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((M, 2 * I), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((M, 2 * I // 32), 98, dtype=torch.uint8, device="cuda")
    nr = None if num_rows is None else torch.tensor([num_rows], dtype=torch.int32, device="cuda")
    g.swiglu_ckpt8(gu.cuda(), h, codes, scales, num_rows=nr)
    torch.cuda.synchronize()
    return h, codes, scales


def check_forward(gu, I, h, codes, scales, slack=0.0):
    v = ref.f64(gu)
    q, sc = ref.ckpt8(v)
    assert np.array_equal(scales.cpu().numpy(), sc), "scale bytes"
    got = ref.decode_ckpt(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(got, q, equal_nan=True), "codes"
    with np.errstate(invalid="ignore", over="ignore"):
        want = v[:, :I] * ref.sigmoid(v[:, :I]) * v[:, I:]
    got = ref.f64(h)
    # above the largest bf16 (and the half step that rounds to it) the value is an infinity of its sign
    big = np.abs(want) >= 2.0 ** 128
    assert np.all(got[big] == np.copysign(np.inf, want[big]))
    ok = np.isfinite(want) & (np.abs(want) < 2.0 ** 128 * (1 - 2.0 ** -9) * (1 - 2.0 ** -20))
    # one rounding to bf16, and exp, division, two products in fp32 (within 2^-20 together); below fp32's normal range absolutely
    assert np.all(np.abs(got - want)[ok] <= (U + 2.0 ** -20 + slack) * np.abs(want)[ok] + 2.0 ** -126)


@pytest.mark.parametrize("M,I", [(1, 32), (3, 96), (7, 160), (1, 2880), (33, 768), (260, 1024), (5, 65536)])
def test_forward(g, M, I):
    gu = bf(inputs.rng(M + I).standard_normal((M, 2 * I)) * 2)
    check_forward(gu, I, *run_forward(g, gu, I))


def test_forward_blocks_of_every_size_and_zero(g):
    """Blocks from the smallest subnormals to the largest values, zero blocks, and a block mixing 40 binades."""
    M, I = 8, 160
    rng = inputs.rng(3)
    a = rng.standard_normal((M, 2 * I))
    for r, s in enumerate([-133, -126, -120, -60, 0, 60, 110, 119]):
        a[r] = np.ldexp(a[r], s)
    a[2, :32] = 0.0
    a[3, 32:64] = -0.0
    a[4, 64:96] = np.ldexp(a[4, 64:96], -np.arange(32))
    gu = bf(a)
    check_forward(gu, I, *run_forward(g, gu, I))


def test_forward_at_gates_whose_sigmoid_is_barely_normal(g):
    """silu(g) u with s between 2^-128 and 2^-120 and an u that brings the product back to ordinary size."""
    I = 32
    a = np.ones((8, 2 * I))
    a[:, :I] = -88.5 + np.arange(8 * I).reshape(8, I) * 0.02
    a[:, I:] = 2.0 ** 100
    gu = bf(a)
    # the exponent -g log2 e < 128 is rounded by up to 2^-18, its constant by 2^-25 relatively: 2^-17 ln 2 in the result
    check_forward(gu, I, *run_forward(g, gu, I), slack=2.0 ** -17)


def test_forward_non_finite_values_spare_their_block(g):
    M, I = 2, 64
    a = inputs.rng(4).standard_normal((M, 2 * I))
    a[0, 3], a[0, 40], a[1, 70] = np.nan, np.inf, -np.inf
    a[1, 96:128] = np.inf
    gu = bf(a)
    h, codes, scales = run_forward(g, gu, I)
    check_forward(gu, I, h, codes, scales)
    assert np.isnan(ref.f64(h)[0, 3])


@pytest.mark.parametrize("n", [0, 1, 6, 9, 50, -3])
def test_forward_rows_past_num_rows_are_left_alone(g, n):
    M, I = 9, 96
    gu = bf(inputs.rng(5).standard_normal((M, 2 * I)))
    live = min(max(n, 0), M)
    h, codes, scales = run_forward(g, gu, I, num_rows=n)
    assert torch.all(h[live:] == 7.0) and torch.all(codes[live:] == 99) and torch.all(scales[live:] == 98)
    if live:
        check_forward(gu[:live], I, h[:live], codes[:live], scales[:live])


@pytest.mark.parametrize("wide", [False, True])
def test_forward_and_backward_past_4_gb(g, wide):
    """A small batch repeated until gate_up and d_gate_up pass 4 GB: every repetition has the small batch's bits.  wide:
    M so large that octets need 64-bit indices, with the live rows at the front (the others are not touched)."""
    rows, I = 96, 2048
    gu = bf(inputs.rng(77).standard_normal((rows, 2 * I)))
    dh = bf(inputs.rng(78).standard_normal((rows, I)))
    small = run_forward(g, gu, I)
    dsmall = torch.empty(rows, 2 * I, dtype=torch.bfloat16, device="cuda")
    g.swiglu_ckpt8_backward(dh.cuda(), small[1], small[2], dsmall)
    n = 3 if wide else 6000  # 6000 * 96 * 4096 * 2 = 4.7e9 bytes
    M = 1 << 23 if wide else n * rows  # 2^23 * 256 octets = 2^31
    tall = lambda t: t.as_strided((M, t.shape[1]), (0, 1)) if wide else t
    nr = torch.tensor([n * rows], dtype=torch.int32, device="cuda") if wide else None
    big = gu.cuda().repeat(n, 1)
    h = torch.full((n * rows + 1, I), 7.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((n * rows + 1, 2 * I), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((n * rows + 1, 2 * I // 32), 98, dtype=torch.uint8, device="cuda")
    cut = lambda t: t if wide else t[:-1]
    g.swiglu_ckpt8(big, tall(cut(h)), codes, scales, num_rows=nr)
    same_rows = lambda t, s: bool((t[:-1].view(n, rows, -1) == s).all())
    assert same_rows(h.view(torch.int16), small[0].view(torch.int16))
    assert same_rows(codes, small[1]) and same_rows(scales, small[2])
    assert torch.all(h[-1] == 7.0) and torch.all(codes[-1] == 99) and torch.all(scales[-1] == 98)
    del big, h
    dbig = dh.cuda().repeat(n, 1)
    d = torch.full((n * rows + 1, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    g.swiglu_ckpt8_backward(tall(dbig), codes, scales, d, num_rows=nr)
    assert same_rows(d.view(torch.int16), dsmall.view(torch.int16)) and torch.all(d[-1] == 7.0)


# ------------------------------------------------------------------------------------------------ backward


def backward_ref(dh, q, I, w):
    """d_gate_up, h, row dots in fp64, and the sums of absolute terms of the dots."""
    gt, u = q[:, :I], q[:, I:]
    s = ref.sigmoid(gt)
    h = gt * s * u
    d = w[:, None] * dh
    return np.concatenate([d * u * s * (1 + gt * (1 - s)), d * gt * s], 1), h, (dh * h).sum(1), np.abs(dh * h).sum(1)


@pytest.mark.parametrize("T,k,I,drop", [(1, 1, 32, 0.0), (1, 8, 96, 0.0), (5, 3, 160, 0.3), (40, 4, 2880, 0.1),
                                        (64, 8, 768, 0.5), (3, 2, 64, 1.0), (2, 2, 16384, 0.0), (700, 8, 32, 0.2)])
@pytest.mark.parametrize("h_out", [False, True])
def test_backward_with_routing(g, T, k, I, drop, h_out):
    M = T * k
    rng = inputs.rng(M * 7 + I)
    s2f, f2s, n = routing(rng, T, k, drop)
    gu = bf(rng.standard_normal((M, 2 * I)) * 2)
    dh = bf(rng.standard_normal((M, I)) * 0.01)
    w = rng.uniform(0.01, 1.0, size=M).astype(np.float32)
    _, codes, scales = run_forward(g, gu, I)
    dgu = torch.full((M, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    h = torch.full((M, I), 7.0, dtype=torch.bfloat16, device="cuda") if h_out else None
    dw = torch.full((T, k), 5.0, device="cuda")
    g.swiglu_ckpt8_backward(dh.cuda(), codes, scales, dgu, sorted_to_flat=dev(s2f), flat_to_sorted=dev(f2s),
                            weights=dev(w), d_weights=dw, h=h,
                            num_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    q = ref.decode_ckpt(codes.cpu().numpy(), scales.cpu().numpy())
    want, wh, dots, mags = backward_ref(ref.f64(dh)[:n], q[:n], I, w[s2f[:n]].astype(np.float64))
    tol = U + 2.0 ** -18  # one rounding; exp, division and six fp32 operations
    # near the zero of silu's slope (1 + g (1 - s) = 0 at g = -1.278) the terms cancel: fp32 steps of the terms
    gt, u = q[:n, :I], q[:n, I:]
    s = ref.sigmoid(gt)
    cancel = np.abs(w[s2f[:n]][:, None] * ref.f64(dh)[:n] * u * s) * (1 + np.abs(gt)) * 2.0 ** -20
    err = np.abs(ref.f64(dgu)[:n] - want)
    assert np.all(err <= tol * np.abs(want) + np.concatenate([cancel, np.zeros_like(cancel)], 1) + 2.0 ** -126)
    assert torch.all(dgu[n:] == 7.0)
    if h_out:
        assert np.all(np.abs(ref.f64(h)[:n] - wh) <= tol * np.abs(wh) + 2.0 ** -126) and torch.all(h[n:] == 7.0)
    want_dw, mag = np.zeros(M), np.zeros(M)
    want_dw[s2f[:n]], mag[s2f[:n]] = dots, mags
    got = dw.cpu().numpy().reshape(-1)
    assert np.all(np.abs(got - want_dw) <= (I * 2.0 ** -24 + 2.0 ** -18) * mag)
    assert np.all(got[f2s < 0] == 0.0)


def test_backward_without_routing_is_the_plain_derivative(g):
    M, I = 37, 224
    rng = inputs.rng(9)
    gu, dh = bf(rng.standard_normal((M, 2 * I))), bf(rng.standard_normal((M, I)))
    _, codes, scales = run_forward(g, gu, I)
    dgu = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    g.swiglu_ckpt8_backward(dh.cuda(), codes, scales, dgu)
    torch.cuda.synchronize()
    q = torch.from_numpy(ref.decode_ckpt(codes.cpu().numpy(), scales.cpu().numpy())).requires_grad_()
    (torch.nn.functional.silu(q[:, :I]) * q[:, I:]).backward(torch.from_numpy(ref.f64(dh)))
    want = q.grad.numpy()
    bound = (U + 2.0 ** -18) * np.abs(want) + 2.0 ** -18 * np.abs(ref.f64(dh).repeat(2, 1).reshape(M, -1)) * 0
    cancel = np.abs(ref.f64(dh) * q.detach().numpy()[:, I:]) * (1 + np.abs(q.detach().numpy()[:, :I])) * 2.0 ** -20
    assert np.all(np.abs(ref.f64(dgu) - want) <= bound + np.concatenate([cancel, cancel * 0], 1))


def test_backward_at_large_gates(g):
    """Saturated gates: silu' is 1 or 0 and nothing turns into NaN."""
    M, I = 2, 64
    a = np.zeros((M, 2 * I))
    a[:, :I] = np.where(np.arange(I) % 2, 1.0, -1.0) * np.logspace(1, 37, I)
    a[:, I:] = 2.0
    gu, dh = bf(a), bf(np.full((M, I), 0.5))
    _, codes, scales = run_forward(g, gu, I)
    dgu = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    g.swiglu_ckpt8_backward(dh.cuda(), codes, scales, dgu)
    torch.cuda.synchronize()
    q = ref.decode_ckpt(codes.cpu().numpy(), scales.cpu().numpy())
    want = backward_ref(ref.f64(dh), q, I, np.ones(M))[0]
    assert np.all(np.abs(ref.f64(dgu) - want) <= (U + 2.0 ** -18) * np.abs(want) + 1e-4 * (np.abs(want) < 1))
    assert np.isfinite(ref.f64(dgu)).all()


# ------------------------------------------------------------------------------------------------ combine, router


@pytest.mark.parametrize("T,k,N,drop", [(1, 1, 8, 0.0), (3, 2, 40, 0.5), (63, 4, 2880, 0.1), (200, 8, 256, 0.0),
                                        (4, 3, 32768, 0.3), (9, 5, 64, 1.0)])
@pytest.mark.parametrize("weighted,with_y", [(True, True), (True, False), (False, True), (False, False)])
def test_combine_backward(g, T, k, N, drop, weighted, with_y):
    M = T * k
    rng = inputs.rng(M + N)
    s2f, f2s, n = routing(rng, T, k, drop)
    dout, y = bf(rng.standard_normal((T, N))), bf(rng.standard_normal((M, N)))
    w = rng.uniform(0.01, 1.0, size=(T, k)).astype(np.float32)
    dy = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), 5.0, device="cuda") if with_y else None
    g.combine_backward(dout.cuda(), dev(s2f), dev(f2s) if with_y else None, dy, k=k, weights=dev(w) if weighted else None,
                       y=y.cuda() if with_y else None, d_weights=dw)
    torch.cuda.synchronize()
    rows = ref.f64(dout)[s2f[:n] // k]
    want = rows * (w.reshape(-1)[s2f[:n]][:, None].astype(np.float64) if weighted else 1.0)
    got = ref.f64(dy)
    assert np.all(np.abs(got[:n] - want) <= (U + 2.0 ** -24) * np.abs(want) * weighted) and np.all(got[n:] == 0.0)
    if with_y:
        ww, mag = np.zeros(M), np.zeros(M)
        prod = rows * ref.f64(y)[:n]
        ww[s2f[:n]], mag[s2f[:n]] = prod.sum(1), np.abs(prod).sum(1)
        d = dw.cpu().numpy().reshape(-1)
        assert np.all(np.abs(d - ww) <= N * 2.0 ** -24 * mag) and np.all(d[f2s < 0] == 0.0)


def test_combine_backward_is_the_gradient_of_combine(g):
    """<combine(y + s), dout> - <combine(y), dout> = <dy, s> (combine is linear), on values where no rounding occurs."""
    T, k, N = 6, 4, 48
    M = T * k
    rng = inputs.rng(17)
    s2f, f2s, n = routing(rng, T, k, 0.25)
    ints = lambda *s: bf(rng.integers(-4, 5, size=s))
    y, step, dout = ints(M, N), ints(M, N), ints(T, N)
    w = dev(rng.choice([0.25, 0.5, 1.0], size=(T, k)).astype(np.float32))
    out = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g.combine(y.cuda(), dev(f2s), w, out[0])
    g.combine((y + step).cuda(), dev(f2s), w, out[1])
    dy = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    g.combine_backward(dout.cuda(), dev(s2f), dev(f2s), dy, k=k, weights=w)
    torch.cuda.synchronize()
    lhs = ((ref.f64(out[1]) - ref.f64(out[0])) * ref.f64(dout)).sum()
    assert lhs == (ref.f64(dy) * ref.f64(step)).sum()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 33, 5), (100, 384, 8), (3, 4096, 32), (50, 70, 32), (9, 130, 1)])
def test_router_backward(g, T, E, k):
    rng = inputs.rng(T + E)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids, p = ref.topk(logits, None, k)
    d = rng.standard_normal((T, k)).astype(np.float32)
    buf = torch.full(((T + 2) * E,), 7.0, device="cuda")
    out = buf[E:(T + 1) * E].view(T, E)
    g.route_topk_backward(dev(ids), dev(p.astype(np.float32)), dev(d), out)
    torch.cuda.synchronize()
    leaf = torch.from_numpy(logits).double().requires_grad_()
    torch.softmax(leaf.gather(1, torch.from_numpy(ids).long()), 1).backward(torch.from_numpy(d).double())
    want = leaf.grad.numpy()
    bound = np.zeros((T, E))  # p is given rounded (2^-24); k products and sums, then a difference and a product
    np.put_along_axis(bound, ids.astype(np.int64), p * (np.abs(d) + (p * np.abs(d)).sum(1, keepdims=True)) * (k + 8) * 2.0 ** -24, 1)
    assert np.all(np.abs(out.cpu().numpy() - want) <= bound)
    assert torch.all(buf[:E] == 7.0) and torch.all(buf[(T + 1) * E:] == 7.0)


def test_router_backward_of_repeated_and_foreign_ids(g):
    ids = np.array([[2, 2, 5, 2], [-1, 0, 9, 3]], np.int32)  # E = 8: -1 and 9 write nothing
    p = np.array([[0.5, 0.25, 0.125, 0.125], [0.25, 0.25, 0.25, 0.25]], np.float32)
    d = np.array([[1.0, 2.0, -4.0, 8.0], [4.0, -4.0, 2.0, 1.0]], np.float32)
    out = torch.empty(2, 8, device="cuda")
    g.route_topk_backward(dev(ids), dev(p), dev(d), out)
    torch.cuda.synchronize()
    want = np.zeros((2, 8))
    for t in range(2):
        s = (p[t] * d[t]).sum()
        for j in range(4):
            if 0 <= ids[t, j] < 8:
                want[t, ids[t, j]] += p[t, j] * (d[t, j] - s)
    assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))  # sums of a few small dyadics: exact


# ------------------------------------------------------------------------------------------------ a whole step


class Step:
    """Forward and backward of a routed layer on MXFP4 stacks through the library, as a training loop makes it."""

    T, E, k, H, I = 24, 6, 2, 128, 96

    def __init__(self, g, seed):
        self.g = g
        T, E, k, H, I = self.T, self.E, self.k, self.H, self.I
        rng = inputs.rng(seed)
        self.w1, self.s1 = inputs.mxfp4_random(rng, E, 2 * I, H, e_lo=119, e_hi=121)
        self.w2, self.s2 = inputs.mxfp4_random(rng, E, H, I, e_lo=119, e_hi=121)
        self.x, self.dout = bf(rng.standard_normal((T, H))), bf(rng.standard_normal((T, H)))
        self.logits = rng.standard_normal((T, E)).astype(np.float32)
        M = T * k
        e = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
        i32 = lambda *s: e(*s, dtype=torch.int32)
        f32 = lambda *s: e(*s, dtype=torch.float32)
        u8 = lambda *s: e(*s, dtype=torch.uint8)
        self.d = {n: dev(getattr(self, n)) for n in ("w1", "s1", "w2", "s2")}
        self.dx_in, self.ddout, self.dlg = self.x.cuda(), self.dout.cuda(), dev(self.logits)
        self.off, self.s2f, self.f2s, self.ids, self.p = i32(E + 1), i32(M), i32(M), i32(T, k), f32(T, k)
        self.xs, self.gu, self.h, self.y, self.out = e(M, H), e(M, 2 * I), e(M, I), e(M, H), e(T, H)
        self.codes, self.scales = u8(M, 2 * I), u8(M, 2 * I // 32)
        self.dys, self.dh, self.dgu, self.dxs, self.dx = e(M, H), e(M, I), e(M, 2 * I), e(M, H), e(T, H)
        self.dw, self.dlogits, self.ones = f32(T, k), f32(T, E), torch.ones(T, k, device="cuda")
        self.ws = u8(max(g.route_workspace_bytes(T, k, E), 16))

    def run(self):
        g, d = self.g, self.d
        n = self.off[self.E:]
        g.route_topk_permute(self.dlg, self.dx_in, self.k, self.ids, self.p, self.off, self.s2f, self.f2s, self.xs, self.ws)
        g.grouped_gemm_mxfp4(self.xs, d["w1"], d["s1"], self.gu, offsets=self.off)
        g.swiglu_ckpt8(self.gu, self.h, self.codes, self.scales, num_rows=n)
        g.grouped_gemm_mxfp4(self.h, d["w2"], d["s2"], self.y, offsets=self.off)
        g.combine(self.y, self.f2s, self.p, self.out)
        g.combine_backward(self.ddout, self.s2f, None, self.dys, k=self.k)
        g.grouped_dgrad_mxfp4(self.dys, d["w2"], d["s2"], self.dh, offsets=self.off)
        g.swiglu_ckpt8_backward(self.dh, self.codes, self.scales, self.dgu, num_rows=n, sorted_to_flat=self.s2f,
                                flat_to_sorted=self.f2s, weights=self.p, d_weights=self.dw)
        g.grouped_dgrad_mxfp4(self.dgu, d["w1"], d["s1"], self.dxs, offsets=self.off)
        g.combine(self.dxs, self.f2s, self.ones, self.dx)
        g.route_topk_backward(self.ids, self.p, self.dw, self.dlogits)

    def dense(self):
        """The layer in fp64 torch, for x and logits: loss = <out, dout>."""
        W1 = torch.from_numpy(np.stack([ref.dequant("mxfp4", self.w1[e], self.s1[e]) for e in range(self.E)]))
        W2 = torch.from_numpy(np.stack([ref.dequant("mxfp4", self.w2[e], self.s2[e]) for e in range(self.E)]))
        ids = self.ids.cpu().long()

        def loss(x, logits):
            p = torch.softmax(logits.gather(1, ids), 1)
            gu = torch.einsum("tkih,th->tki", W1[ids], x)
            h = torch.nn.functional.silu(gu[..., :self.I]) * gu[..., self.I:]
            y = torch.einsum("tkhi,tki->tkh", W2[ids], h)
            return (torch.einsum("tk,tkh->th", p, y) * torch.from_numpy(ref.f64(self.dout))).sum()

        return loss


def rel(a, b):
    return float(np.sqrt(((a - b) ** 2).sum() / (b ** 2).sum()))


def test_a_training_step_against_the_formulas_gradient_and_differences(g):
    st = Step(g, 5)
    st.run()
    torch.cuda.synchronize()
    loss = st.dense()
    x = torch.from_numpy(ref.f64(st.x)).requires_grad_()
    lg = torch.from_numpy(st.logits.astype(np.float64)).requires_grad_()
    v = loss(x, lg)
    v.backward()
    # e4m3 keeps 4 significant bits: an element is off by at most 2^-4, 2^-4 / sqrt(3) = 0.036 in the mean, g and u
    # independently; a factor of 2 for the activation's slope (silu' changes by up to 0.5 per unit of g) on g of size 1-2
    tol = 2 * 2.0 ** -4 * (2 / 3) ** 0.5
    assert rel(ref.f64(st.dx), x.grad.numpy()) <= tol
    assert rel(ref.f64(st.dlogits), lg.grad.numpy()) <= tol
    # against differences of the fp64 loss along random directions, to the same tolerance of the derivative's size
    rng = inputs.rng(6)
    for leaf, got in ((x, ref.f64(st.dx)), (lg, ref.f64(st.dlogits))):
        step = torch.from_numpy(rng.standard_normal(tuple(leaf.shape)))
        eps = 1e-5
        args = lambda s: (x.detach() + s * step, lg.detach()) if leaf is x else (x.detach(), lg.detach() + s * step)
        diff = float((loss(*args(eps)) - loss(*args(-eps))) / (2 * eps))
        assert abs(diff - float((got * step.numpy()).sum())) <= 4 * tol * np.sqrt((leaf.grad.numpy() ** 2).sum())
    out = float((ref.f64(st.out) * ref.f64(st.dout)).sum())
    # forward: y, h and out are rounded to bf16 (three times 2^-8 / sqrt(3)), gate_up once (silu's slope doubles it)
    assert abs(out - float(v)) <= 4 * 2.0 ** -8 * 5 ** 0.5 * float(np.sqrt((ref.f64(st.out) ** 2).sum() * (ref.f64(st.dout) ** 2).mean()))


def test_the_step_is_repeatable_captured_and_matches_the_decode_call(g):
    st = Step(g, 8)
    st.run()
    torch.cuda.synchronize()
    names = ("out", "dx", "dlogits", "dw", "dgu", "codes", "scales")
    first = {n: getattr(st, n).clone() for n in names}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for n in names:
        getattr(st, n).zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n in names:
        assert same(first[n], getattr(st, n)), n
    # eight of its tokens through the whole-layer call on the same stacks
    T, k, H, I, E = 8, st.k, st.H, st.I, st.E
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ids, p = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    ws = torch.zeros(g.moe_decode_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    g.moe_decode_mxfp4(st.dx_in[:T], st.d["w1"], st.d["s1"], st.d["w2"], st.d["s2"], st.dlg[:T], ids, p, out, ws)
    torch.cuda.synchronize()
    assert torch.equal(ids, st.ids[:T])
    # the step rounds gate_up, h, y and out, the call p*h and out
    assert rel(ref.f64(out), ref.f64(st.out[:T])) <= 2.0 ** -8 * 8 ** 0.5


def test_every_call_on_another_stream(g):
    st = Step(g, 12)
    st.run()
    torch.cuda.synchronize()
    want = {n: getattr(st, n).clone() for n in ("out", "dx", "dlogits")}
    side = torch.cuda.Stream()
    for n in want:
        getattr(st, n).zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        st.run()
    side.synchronize()
    for n, v in want.items():
        assert same(v, getattr(st, n))
