"""gnf4_moe_decode_{nf4,mxfp4}: a whole routed layer for up to 8 tokens in one launch, against the 64-bit definition
(tests/_layer_ref.py derives the bound), the routing call's selection, and itself: repeated, captured, on other
streams, with a workspace used by several shapes."""
import numpy as np
import pytest
import torch

from bit_grouped_moe_b200 import inputs
from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from bit_grouped_moe_b200 import gnf4
    gnf4.device_errors(clear=True)
    yield gnf4
    assert gnf4.device_errors() == 0


def stack(fmt, E, N, K, seed):
    rng = inputs.rng(seed)
    if fmt == "nf4":
        w = rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8)
        return w, (0.05 * rng.uniform(0.3, 1.5, size=(E, N, K // 64))).astype(np.float32)
    return inputs.mxfp4_random(rng, E, N, K, e_lo=118, e_hi=122)


def same_bits(a, b):
    v = lambda t: t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()
    return bool(np.array_equal(v(a), v(b)))


class Layer:
    """Inputs and outputs of one call, the outputs inside larger guarded buffers."""

    def __init__(self, g, fmt, T, E, k, H, I, router=True, bias=False, seed=0, workspace=None):
        self.g, self.fmt, self.T, self.E, self.k, self.H, self.I = g, fmt, T, E, k, H, I
        rng = inputs.rng(seed + 7)
        self.w1, self.s1 = stack(fmt, E, 2 * I, H, seed + 1)
        self.w2, self.s2 = stack(fmt, E, H, I, seed + 2)
        self.x = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).bfloat16()
        self.router = (torch.from_numpy(rng.standard_normal((E, H), dtype=np.float32)) * H ** -0.5).bfloat16() if router else None
        self.bias = (rng.standard_normal(E, dtype=np.float32) * np.float32(0.5)) if bias else None
        self.logits_in = None if router else rng.standard_normal((T, E), dtype=np.float32)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.d = {n: dev(getattr(self, n)) for n in ("w1", "s1", "w2", "s2")}
        self.dx = self.x.cuda()
        self.drouter = None if self.router is None else self.router.cuda()
        self.dbias = None if self.bias is None else dev(self.bias)
        self.logits = torch.full((T, E), 3.5, device="cuda") if router else dev(self.logits_in)
        self.guard = torch.full(((T + 2) * H,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.out = self.guard[H:(T + 1) * H].view(T, H)
        self.gid = torch.full(((T + 2) * k,), -9, dtype=torch.int32, device="cuda")
        self.ids = self.gid[k:(T + 1) * k].view(T, k)
        self.gp = torch.full(((T + 2) * k,), -9.0, device="cuda")
        self.p = self.gp[k:(T + 1) * k].view(T, k)
        self.ws = workspace if workspace is not None else self.new_workspace()

    def new_workspace(self):
        return torch.zeros(self.g.moe_decode_workspace_bytes(self.T, self.k, self.H, self.I), dtype=torch.uint8,
                           device="cuda")

    def call(self, stream=None):
        f = self.g.moe_decode_nf4 if self.fmt == "nf4" else self.g.moe_decode_mxfp4
        f(self.dx, self.d["w1"], self.d["s1"], self.d["w2"], self.d["s2"], self.logits, self.ids, self.p, self.out,
          self.ws, router_w=self.drouter, bias=self.dbias, stream=stream)

    def result(self):
        torch.cuda.synchronize()
        assert self.g.device_errors() == 0
        return self.out.clone(), self.ids.clone(), self.p.clone(), self.logits.clone()

    def check(self):
        out, ids, p, logits = self.result()
        x = ref.f64(self.x)
        if self.router is not None:
            lg = x @ ref.f64(self.router).T
            mag = np.abs(x) @ np.abs(ref.f64(self.router)).T
            assert np.all(np.abs(logits.cpu().numpy() - lg) <= (self.H + 8) * 2.0 ** -24 * mag + 1e-30), "logits"
        want_ids, want_p = ref.topk(logits.cpu().numpy(), self.bias, self.k)
        assert np.array_equal(ids.cpu().numpy(), want_ids), "topk_ids"
        # expf and the division are within a few units of 2^-23; k terms are added
        assert np.all(np.abs(p.cpu().numpy() - want_p) <= (self.k + 16) * 2.0 ** -24 * want_p + 1e-37), "topk_weights"
        want, bound = ref.layer(self.fmt, x, want_ids, want_p, self.w1, self.s1, self.w2, self.s2)
        err = np.abs(ref.f64(out) - want)
        assert np.all(err <= bound), f"worst error / bound {np.nanmax(err / bound):.3g}"
        # independent roundings (out, h, two NF4 codes), each at most 2^-8 and evenly spread: 2^-8 sqrt(4/3) in the mean
        rms = np.sqrt((err ** 2).mean() / (want ** 2).mean())
        assert rms <= 2.0 ** -8 * (4 / 3) ** 0.5, rms
        assert torch.all(self.guard[:self.H] == 7.0) and torch.all(self.guard[(self.T + 1) * self.H:] == 7.0)
        assert torch.all(self.gid[:self.k] == -9) and torch.all(self.gid[(self.T + 1) * self.k:] == -9)
        assert torch.all(self.gp[:self.k] == -9) and torch.all(self.gp[(self.T + 1) * self.k:] == -9)


SHAPES = [
    # fmt, T, E, k, H, I
    ("mxfp4", 1, 1, 1, 32, 32), ("nf4", 1, 1, 1, 64, 64), ("nf4", 1, 8, 2, 256, 128), ("mxfp4", 1, 8, 2, 256, 128),
    ("mxfp4", 3, 5, 3, 96, 160), ("nf4", 7, 6, 4, 192, 448), ("mxfp4", 8, 16, 8, 480, 96), ("nf4", 8, 16, 16, 320, 64),
    ("nf4", 2, 64, 8, 2048, 1024), ("mxfp4", 5, 12, 4, 2880, 2880), ("nf4", 8, 40, 8, 1024, 768),
    ("mxfp4", 8, 4, 2, 7168, 256), ("mxfp4", 4, 300, 32, 128, 64), ("nf4", 8, 64, 32, 128, 64),
]


@pytest.mark.parametrize("fmt,T,E,k,H,I", SHAPES)
@pytest.mark.parametrize("router,bias", [(True, False), (False, True)])
def test_layer_against_the_definition(g, fmt, T, E, k, H, I, router, bias):
    lay = Layer(g, fmt, T, E, k, H, I, router=router, bias=bias, seed=T * 131 + H)
    lay.call()
    lay.check()


@pytest.mark.parametrize("fmt,T,E,k,H,I", [("mxfp4", 1, 2, 1, 57344, 64), ("nf4", 1, 2, 2, 64, 65536),
                                           ("mxfp4", 2, 1024, 8, 64, 32), ("nf4", 7, 2, 1, 8192, 64)])
def test_layer_at_the_documented_limits(g, fmt, T, E, k, H, I):
    lay = Layer(g, fmt, T, E, k, H, I, seed=11)
    lay.call()
    lay.check()


@pytest.mark.parametrize("bias", [False, True])
def test_selection_is_the_routing_calls(g, bias):
    """Ties, signed zeros, infinities and NaN: ids and weights equal gnf4_route_topk_permute's bit for bit."""
    T, E, k, H = 8, 70, 9, 64
    lay = Layer(g, "nf4", T, E, k, H, 64, router=False, bias=bias, seed=3)
    lg = inputs.rng(5).integers(-3, 4, size=(T, E)).astype(np.float32)  # many ties
    lg[1] = 0.0
    lg[1, ::2] = -0.0
    lg[2, :65] = np.nan
    lg[3, :66] = -np.inf
    lg[4, 5] = np.inf
    lg[5] = np.nan
    lay.logits.copy_(torch.from_numpy(lg))
    lay.call()
    _, ids, p, logits = lay.result()
    assert np.array_equal(logits.cpu().numpy(), lg, equal_nan=True)  # an input
    M = T * k
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    rid, rp = i32(M).view(T, k), torch.empty(T, k, device="cuda")
    ws = torch.empty(max(g.route_workspace_bytes(T, k, E), 16), dtype=torch.uint8, device="cuda")
    g.route_topk_permute(lay.logits, lay.dx, k, rid, rp, i32(E + 1), i32(M), i32(M),
                         torch.empty(M, H, dtype=torch.bfloat16, device="cuda"), ws, bias=lay.dbias)
    torch.cuda.synchronize()
    assert torch.equal(ids, rid)
    assert torch.equal(p.view(torch.int32)[~torch.isnan(rp)], rp.view(torch.int32)[~torch.isnan(rp)])
    assert torch.equal(torch.isnan(p), torch.isnan(rp))


def test_a_tokens_nan_and_infinity_stay_in_its_row(g):
    lay = Layer(g, "mxfp4", 6, 12, 4, 256, 160, router=False, seed=21)
    lay.call()
    clean = lay.result()[0]
    lay.dx[2, 17] = float("nan")
    lay.dx[4, 3] = float("inf")
    lay.call()
    out = lay.result()[0]
    keep = [0, 1, 3, 5]
    assert same_bits(out[keep], clean[keep])
    assert torch.isnan(out[2]).all() and not torch.isfinite(out[4]).any()


def test_nan_scale_of_an_expert_reaches_the_tokens_that_chose_it(g):
    lay = Layer(g, "mxfp4", 4, 6, 2, 128, 64, router=False, seed=23)
    lay.call()
    clean, ids = lay.result()[:2]
    e = int(ids[0, 0])
    lay.d["s2"][e] = 255  # e8m0 NaN
    lay.call()
    out = lay.result()[0]
    hit = (ids == e).any(dim=1)
    assert torch.isnan(out[hit]).all()
    assert same_bits(out[~hit], clean[~hit])


@pytest.mark.parametrize("lo,hi,xs", [(0, 3, 2.0 ** 60), (126, 132, 2.0 ** -3), (180, 190, 2.0 ** -60), (250, 251, 2.0 ** -125)])
def test_mxfp4_scales_over_their_range(g, lo, hi, xs):
    """Scale bytes from the smallest to the largest whose decoded weights are finite."""
    lay = Layer(g, "mxfp4", 2, 3, 2, 128, 96, router=False, seed=29)
    rng = inputs.rng(31)
    lay.s1 = rng.integers(lo, hi + 1, size=lay.s1.shape, dtype=np.uint8)
    lay.d["s1"].copy_(torch.from_numpy(lay.s1))
    lay.x = (lay.x.float() * xs).bfloat16()
    lay.dx.copy_(lay.x)
    lay.call()
    lay.check()


def test_repeated_calls_give_the_same_bits_and_leave_the_workspace_ready(g):
    big = Layer(g, "nf4", 8, 32, 8, 1024, 512, seed=41)
    small = Layer(g, "mxfp4", 3, 8, 2, 96, 64, seed=43, workspace=big.ws)
    wide = Layer(g, "mxfp4", 1, 4, 2, 8192, 64, seed=47, workspace=big.ws)
    big.call()
    first = big.result()
    for _ in range(20):
        small.call()
        wide.call()
        big.call()
    again = big.result()
    for a, b in zip(first, again):
        assert same_bits(a, b)
    small.check()
    wide.check()
    big.check()


def test_captured_and_replayed_with_a_shared_workspace(g):
    a = Layer(g, "nf4", 4, 16, 4, 512, 256, seed=51)
    b = Layer(g, "mxfp4", 2, 16, 4, 480, 96, seed=53, workspace=a.ws)
    a.call()
    b.call()
    want = a.result()[0], b.result()[0]
    graphs = []
    for lay in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            lay.call()
        graphs.append(gr)
    for lay in (a, b):
        lay.out.fill_(9.0)
    for _ in range(5):
        for gr in graphs:
            gr.replay()
    for lay, w in zip((a, b), want):
        assert same_bits(lay.result()[0], w)
    # new inputs in the captured buffers
    a.x = (a.x.float() * 0.5).bfloat16()
    a.dx.copy_(a.x)
    graphs[0].replay()
    a.check()


def test_two_streams_at_once_with_a_workspace_each(g):
    lays = [Layer(g, f, T, 24, 6, 1024, 512, seed=61 + T) for f, T in (("nf4", 8), ("mxfp4", 5))]
    streams = [torch.cuda.Stream() for _ in lays]
    torch.cuda.synchronize()
    for _ in range(30):
        for lay, st in zip(lays, streams):
            lay.call(stream=st)
    for lay in lays:
        lay.check()


def test_agrees_with_the_separate_calls(g):
    """route_topk_permute, gemv_swiglu and gemv_combine on the same stacks: equal within both sides' rounding."""
    T, E, k, H, I = 6, 16, 4, 512, 256
    lay = Layer(g, "mxfp4", T, E, k, H, I, router=False, seed=71)
    lay.call()
    out = lay.result()[0]
    M = T * k
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    off, s2f, f2s = i32(E + 1), i32(M), i32(M)
    ids, p, xs, h, y, out2 = i32(M).view(T, k), torch.empty(T, k, device="cuda"), bf(M, H), bf(M, I), bf(M, H), bf(T, H)
    ws = torch.empty(max(g.route_workspace_bytes(T, k, E), 16), dtype=torch.uint8, device="cuda")
    cnt = torch.zeros(g.combine_counters_bytes(T, H), dtype=torch.uint8, device="cuda")
    g.route_topk_permute(lay.logits, lay.dx, k, ids, p, off, s2f, f2s, xs, ws)
    g.grouped_gemv_mxfp4_swiglu(xs, lay.d["w1"], lay.d["s1"], h, offsets=off)
    g.grouped_gemv_mxfp4_combine(h, lay.d["w2"], lay.d["s2"], y, s2f, f2s, p, out2, cnt, offsets=off)
    torch.cuda.synchronize()
    want, bound = ref.layer("mxfp4", ref.f64(lay.x), ids.cpu().numpy(), ref.f64(p), lay.w1, lay.s1, lay.w2, lay.s2)
    # the separate calls also round every expert's output y: one more 2^-8 of sum_j p |y_j|, which the bound's own
    # h term (2^-8 of sum |D||h|) dominates
    assert np.all(np.abs(ref.f64(out) - ref.f64(out2)) <= 3 * bound)


def test_no_tokens(g):
    lay = Layer(g, "nf4", 1, 4, 2, 64, 64, seed=81)
    g.call_stats_get("gnf4_moe_decode_nf4", reset=True)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    g.moe_decode_nf4(e, lay.d["w1"], lay.d["s1"], lay.d["w2"], lay.d["s2"], lay.logits[:0], lay.ids[:0], lay.p[:0], e,
                     lay.ws)
    lay.call()
    torch.cuda.synchronize()
    s = g.call_stats_get("gnf4_moe_decode_nf4")
    assert (s["calls"], s["engaged"], s["rows"]) == (2, 1, 2)


def test_short_or_misaligned_workspace_is_refused_before_any_launch(g):
    lay = Layer(g, "mxfp4", 2, 4, 2, 64, 64, seed=91)
    lay.out.fill_(7.0)
    for ws in (lay.ws[:-1], lay.ws[:0], torch.zeros(lay.ws.numel() + 8, dtype=torch.uint8, device="cuda")[8:]):
        lay.ws = ws
        with pytest.raises(g.Gnf4Error) as e:
            lay.call()
        assert e.value.status == g.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.all(lay.out == 7.0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nf4"])
def test_the_last_experts_of_stacks_past_4_gb(g, fmt):
    """Experts placed at the end of stacks of 5.6 and 2.8 GB give the bits that the same experts give in a small stack."""
    T, few, E, k, H, I = 3, 6, 384, 4, 7168, 2048
    lay = Layer(g, fmt, T, few, k, H, I, router=False, seed=101)
    lay.call()
    want = lay.result()
    for n in ("w1", "s1", "w2", "s2"):
        part = lay.d[n]
        lay.d[n] = torch.zeros((E,) + part.shape[1:], dtype=part.dtype, device="cuda")
        lay.d[n][E - few:] = part
    small = lay.logits
    lay.logits = torch.full((T, E), -1e30, device="cuda")
    lay.logits[:, E - few:] = small
    lay.call()
    out, ids, p, _ = lay.result()
    assert torch.equal(ids, want[1] + (E - few)) and same_bits(p, want[2])
    assert same_bits(out, want[0])
