"""Timed cases of the Mixture-of-Experts layer operators.

``decode``        gnf4_moe_decode_{nf4,mxfp4}: a whole routed layer for 1 to 8 tokens (router product, top-k,
                  gate_up, SwiGLU, down, weighted sum) on the packed expert stacks.
``step``          gnf4_swiglu_ckpt8 and gnf4_swiglu_ckpt8_backward: the activation of a training step that keeps
                  gate_up in 8 bits (e4m3 codes, one e8m0 scale per 32), and its backward pass from those bits,
                  with the gradient of the router weights.
``combine_bwd``   gnf4_combine_backward: the gradient of the top-k weighted sum.
``router_bwd``    gnf4_route_topk_backward: the gradient of the router's top-k softmax.

A state holds inputs and preallocated outputs; ``run`` makes one pass, in elementary torch operations or (``own``)
through the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# NormalFloat-4 code values (QLoRA) and OCP e2m1 values, by nibble.
NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
       -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
       0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
BLOCK = {"nf4": 64, "mxfp4": 32}


def listed():
    """Sizes of the repository's workloads (OLMoE, Qwen3-30B-A3B, gpt-oss-120b, Kimi-class shapes)."""
    return [
        # one token of one user: latency; 8 experts of 2048 x 2048 and 2048 x 1024
        {"name": "decode-nf4-t1", "op": "decode", "fmt": "nf4", "T": 1, "E": 64, "k": 8, "H": 2048, "I": 1024,
         "router": True, "bias": False},
        # eight users' tokens together: most experts are hit by one or two tokens each
        {"name": "decode-nf4-t8", "op": "decode", "fmt": "nf4", "T": 8, "E": 64, "k": 8, "H": 2048, "I": 1024,
         "router": True, "bias": False},
        # a few speculated tokens behind a router of the model's own (logits given)
        {"name": "decode-nf4-t5-logits", "op": "decode", "fmt": "nf4", "T": 5, "E": 128, "k": 8, "H": 2048, "I": 768,
         "router": False, "bias": False},
        # one token, wide experts, a width that is no multiple of 128
        {"name": "decode-mxfp4-t1", "op": "decode", "fmt": "mxfp4", "T": 1, "E": 128, "k": 4, "H": 2880, "I": 2880,
         "router": True, "bias": False},
        # the heaviest decode step: eight tokens over 48 large experts, selection bias (load balancing)
        {"name": "decode-mxfp4-t8", "op": "decode", "fmt": "mxfp4", "T": 8, "E": 48, "k": 8, "H": 7168, "I": 2048,
         "router": True, "bias": True},
        # a fine-tuning step on a handful of rows
        {"name": "step-small", "op": "step", "T": 9, "k": 8, "I": 1024, "drop": 0.0, "h_out": False},
        # a fine-tuning step of 2048 tokens; a quarter of the experts live elsewhere (their pairs are dropped);
        # h is recomputed for an adapter on the down projection
        {"name": "step-mid", "op": "step", "T": 2048, "k": 8, "I": 768, "drop": 0.25, "h_out": True},
        # a fine-tuning step of 4096 tokens
        {"name": "step-large", "op": "step", "T": 4096, "k": 8, "I": 2048, "drop": 0.0, "h_out": False},
        # backward of the weighted sum: a short sequence, and a full batch with kept expert outputs
        {"name": "combine-bwd-small", "op": "combine_bwd", "T": 63, "k": 4, "N": 2880, "y": True, "weighted": True,
         "drop": 0.1},
        {"name": "combine-bwd-large", "op": "combine_bwd", "T": 2048, "k": 8, "N": 2048, "y": True, "weighted": True,
         "drop": 0.0},
        # gradient of the router's selection: a short sequence, and a full batch over 384 experts
        {"name": "router-bwd-small", "op": "router_bwd", "T": 64, "E": 128, "k": 4},
        {"name": "router-bwd-large", "op": "router_bwd", "T": 4096, "E": 384, "k": 8},
    ]


def _log_int(rng, lo, hi, mult=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / mult)) * mult))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "step", "step", "combine_bwd", "router_bwd"])
    if op == "decode":
        fmt = rng.choice(["nf4", "mxfp4"])
        b = BLOCK[fmt]
        E = rng.choice([8, 16, 48, 64, 128])
        H, I = _log_int(rng, 128, 7168, b), _log_int(rng, 64, 2880, b)
        while E * H * I > 128 * 2880 * 2880:  # no stack above the listed ones
            E //= 2
        return {"op": op, "fmt": fmt, "T": rng.randint(1, 8), "E": E, "k": rng.randint(1, 8), "H": H, "I": I,
                "router": rng.random() < 0.75, "bias": rng.random() < 0.5}
    if op == "step":
        return {"op": op, "T": _log_int(rng, 1, 4096), "k": rng.randint(1, 8), "I": _log_int(rng, 32, 2048, 32),
                "drop": rng.choice([0.0, 0.1, 0.5]), "h_out": rng.random() < 0.5}
    if op == "combine_bwd":
        return {"op": op, "T": _log_int(rng, 1, 2048), "k": rng.randint(1, 8), "N": _log_int(rng, 64, 2048, 8),
                "y": rng.random() < 0.6, "weighted": rng.random() < 0.6, "drop": rng.choice([0.0, 0.1, 0.5])}
    E = _log_int(rng, 8, 384)
    return {"op": op, "T": _log_int(rng, 1, 4096), "E": E, "k": rng.randint(1, min(E, 8))}


# ---------------------------------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _stack(g, fmt, E, N, K):
    """A packed expert stack: codes uniform over the 16, scales as weights of about 0.02 would carry."""
    w = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
    if fmt == "nf4":  # the largest of 64 normal draws, near 2.4 standard deviations
        s = 0.02 * (2.4 + 0.4 * torch.randn(E, N, K // 64, generator=g, device="cuda")).clamp_(1.0, 4.0)
    else:
        s = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda").random_(119, 122, generator=g)
    return w, s


def _routing(g, T, k, drop):
    """Pairs sorted by expert, as the routing calls leave them: sorted_to_flat and flat_to_sorted (-1: none)."""
    E = 64
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(dim=1)[:, :k].reshape(-1)
    ids = torch.where(torch.rand(T * k, generator=g, device="cuda") < drop, E, ids)  # E: an expert held elsewhere
    order = torch.argsort(ids, stable=True)
    n = (ids < E).sum()
    live = torch.arange(T * k, device="cuda") < n
    s2f = torch.where(live, order, -1)
    f2s = torch.empty_like(order)
    f2s[order] = torch.where(live, torch.arange(T * k, device="cuda"), -1)
    weights = torch.softmax(_randn(g, T, k), dim=1)
    return s2f.int(), f2s.int(), n.int().reshape(1), weights


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dev = {"device": "cuda"}
    if case["op"] == "decode":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["w1"], s["s1"] = _stack(g, case["fmt"], E, 2 * I, H)
        s["w2"], s["s2"] = _stack(g, case["fmt"], E, H, I)
        s["x"] = _randn(g, T, H).bfloat16()
        s["router_w"] = _randn(g, E, H, std=H ** -0.5).bfloat16() if case["router"] else None
        s["bias"] = _randn(g, E, std=0.3) if case["bias"] else None
        s["logits"] = torch.zeros(T, E, **dev) if case["router"] else _randn(g, T, E)
        s["codes"] = torch.tensor(NF4 if case["fmt"] == "nf4" else E2M1, **dev)
        s["ids"] = torch.zeros(T, k, dtype=torch.int32, **dev)
        s["wts"] = torch.zeros(T, k, **dev)
        s["out"] = torch.zeros(T, H, dtype=torch.bfloat16, **dev)
        if own:
            from bit_grouped_moe_b200 import gnf4
            s["workspace"] = torch.zeros(gnf4.moe_decode_workspace_bytes(T, k, H, I), dtype=torch.uint8, **dev)
    elif case["op"] == "step":
        T, k, I = case["T"], case["k"], case["I"]
        M = T * k
        s["s2f"], s["f2s"], s["n"], s["weights"] = _routing(g, T, k, case["drop"])
        s["gate_up"] = _randn(g, M, 2 * I, std=1.5).bfloat16()
        s["dh"] = _randn(g, M, I, std=1e-2).bfloat16()
        s["h"] = torch.zeros(M, I, dtype=torch.bfloat16, **dev)
        s["d_gate_up"] = torch.zeros(M, 2 * I, dtype=torch.bfloat16, **dev)
        s["h2"] = torch.zeros(M, I, dtype=torch.bfloat16, **dev) if case["h_out"] else None
        s["d_weights"] = torch.zeros(T, k, **dev)
        if own:
            s["codes"] = torch.zeros(M, 2 * I, dtype=torch.uint8, **dev)
            s["scales"] = torch.zeros(M, 2 * I // 32, dtype=torch.uint8, **dev)
    elif case["op"] == "combine_bwd":
        T, k, N = case["T"], case["k"], case["N"]
        s["s2f"], s["f2s"], s["n"], weights = _routing(g, T, k, case["drop"])
        s["weights"] = weights if case["weighted"] else None
        s["dout"] = _randn(g, T, N, std=1e-2).bfloat16()
        s["y"] = _randn(g, T * k, N).bfloat16() if case["y"] else None
        s["dy"] = torch.zeros(T * k, N, dtype=torch.bfloat16, **dev)
        s["d_weights"] = torch.zeros(T, k, **dev) if case["y"] else None
    else:
        T, E, k = case["T"], case["E"], case["k"]
        logits = _randn(g, T, E)
        s["ids"] = logits.argsort(dim=1, descending=True)[:, :k].int().contiguous()
        s["wts"] = torch.softmax(logits.gather(1, s["ids"].long()), dim=1)
        s["d_weights"] = _randn(g, T, k, std=1e-2)
        s["d_logits"] = torch.zeros(T, E, **dev)
    return s


# ---------------------------------------------------------------------------------------------------- one pass


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _dequant(fmt, codes, w, scales):
    """One expert's packed rows [N, K/2] as fp32 [N, K]."""
    N, K = w.shape[0], 2 * w.shape[1]
    hi, lo = (w >> 4).long(), (w & 15).long()
    pair = torch.stack((hi, lo) if fmt == "nf4" else (lo, hi), dim=-1)
    if fmt != "nf4":
        scales = torch.exp2(scales.float() - 127.0)
    return (codes[pair].view(N, K // BLOCK[fmt], BLOCK[fmt]) * scales[..., None]).view(N, K)


def _decode_plain(s):
    T, k, I = s["T"], s["k"], s["I"]
    if s["router"]:  # 64-bit sums: the selection stands next to a border
        s["logits"].copy_(s["x"].double() @ s["router_w"].double().t())
    logits = s["logits"]
    score = logits if s["bias"] is None else logits + s["bias"]
    ids = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k]
    sel = logits.gather(1, ids)
    e = torch.exp(sel - sel.amax(dim=1, keepdim=True))
    wts = e / e.sum(dim=1, keepdim=True)
    rows = []
    for t in range(T):
        x = s["x"][t].float()
        acc = 0.0
        for j in range(k):
            i = ids[t, j:j + 1]
            gu = _dequant(s["fmt"], s["codes"], s["w1"].index_select(0, i)[0], s["s1"].index_select(0, i)[0]) @ x
            h = gu[:I] / (1.0 + torch.exp(-gu[:I])) * gu[I:]
            y = _dequant(s["fmt"], s["codes"], s["w2"].index_select(0, i)[0], s["s2"].index_select(0, i)[0]) @ h
            acc = acc + wts[t, j] * y
        rows.append(acc)
    return _decode_outputs(s, torch.stack(rows).bfloat16(), ids.int(), wts, logits)


def _decode_outputs(s, out, ids, wts, logits):
    got = {"out": out, "topk_ids": ids, "topk_weights": wts}
    if s["router"]:  # else the logits are an input
        got["logits"] = logits
    return got


def _decode_own(s):
    from bit_grouped_moe_b200 import gnf4
    call = gnf4.moe_decode_nf4 if s["fmt"] == "nf4" else gnf4.moe_decode_mxfp4
    call(s["x"], s["w1"], s["s1"], s["w2"], s["s2"], s["logits"], s["ids"], s["wts"], s["out"], s["workspace"],
         router_w=s["router_w"], bias=s["bias"])
    return _decode_outputs(s, s["out"], s["ids"], s["wts"], s["logits"])


def _ckpt8(v):
    """bf16 [M, C] through e4m3 with one power-of-two scale per 32: 2^(floor(log2(max)) - 7), at least 2^-127."""
    b = v.float().view(v.shape[0], -1, 32)
    ex = torch.frexp(b.abs().amax(dim=-1, keepdim=True)).exponent - 8
    ex = torch.where(b.abs().amax(dim=-1, keepdim=True) > 0, ex, -127).clamp(min=-127)
    q = torch.ldexp(b, -ex).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, ex).view(v.shape)


def _step_plain(s):
    M, I = s["gate_up"].shape[0], s["I"]
    live = (s["s2f"] >= 0)[:, None]
    gu = s["gate_up"].float()
    h = torch.where(live, gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:], 0.0).bfloat16()
    q = _ckpt8(s["gate_up"])
    g, u = q[:, :I], q[:, I:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    hq = g * sig * u
    dh = s["dh"].float()
    w = s["weights"].view(-1)[s["s2f"].clamp(min=0).long()][:, None]
    d = w * dh
    dgu = torch.cat((d * u * sig * (1.0 + g * (1.0 - sig)), d * g * sig), dim=1)
    rows = (dh * hq).sum(dim=1)
    dw = torch.where(s["f2s"] >= 0, rows[s["f2s"].clamp(min=0).long()], 0.0).view_as(s["weights"])
    out = {"h": h, "d_gate_up": torch.where(live, dgu, 0.0).bfloat16(), "d_weights": dw}
    if s["h_out"]:
        out["h2"] = torch.where(live, hq, 0.0).bfloat16()
    return out


def _step_own(s):
    from bit_grouped_moe_b200 import gnf4
    gnf4.swiglu_ckpt8(s["gate_up"], s["h"], s["codes"], s["scales"], num_rows=s["n"])
    gnf4.swiglu_ckpt8_backward(s["dh"], s["codes"], s["scales"], s["d_gate_up"], num_rows=s["n"],
                               sorted_to_flat=s["s2f"], flat_to_sorted=s["f2s"], weights=s["weights"],
                               d_weights=s["d_weights"], h=s["h2"])
    out = {"h": s["h"], "d_gate_up": s["d_gate_up"], "d_weights": s["d_weights"]}
    if s["h_out"]:
        out["h2"] = s["h2"]
    return out


def _combine_bwd_plain(s):
    k = s["k"]
    live = s["s2f"] >= 0
    f = s["s2f"].clamp(min=0).long()
    rows = s["dout"].float()[f // k]
    dy = rows if s["weights"] is None else rows * s["weights"].view(-1)[f][:, None]
    out = {"dy": torch.where(live[:, None], dy, 0.0).bfloat16()}
    if s["y"] is not None:
        dots = (rows * s["y"].float()).sum(dim=1)
        out["d_weights"] = torch.where(s["f2s"] >= 0, dots[s["f2s"].clamp(min=0).long()], 0.0).view(-1, k)
    return out


def _combine_bwd_own(s):
    from bit_grouped_moe_b200 import gnf4
    gnf4.combine_backward(s["dout"], s["s2f"], s["f2s"], s["dy"], k=s["k"], weights=s["weights"], y=s["y"],
                          d_weights=s["d_weights"])
    return {"dy": s["dy"]} if s["y"] is None else {"dy": s["dy"], "d_weights": s["d_weights"]}


def _router_bwd_plain(s):
    p, dw = s["wts"], s["d_weights"]
    d = p * (dw - (p * dw).sum(dim=1, keepdim=True))
    return torch.zeros(s["T"], s["E"], device="cuda").scatter(1, s["ids"].long(), d)


def _router_bwd_own(s):
    from bit_grouped_moe_b200 import gnf4
    gnf4.route_topk_backward(s["ids"], s["wts"], s["d_weights"], s["d_logits"])
    return s["d_logits"]


_plain = {"decode": _decode_plain, "step": _step_plain, "combine_bwd": _combine_bwd_plain,
          "router_bwd": _router_bwd_plain}
_own = {"decode": _decode_own, "step": _step_own, "combine_bwd": _combine_bwd_own, "router_bwd": _router_bwd_own}


# ---------------------------------------------------------------------------------------------------- work


def work(case):
    if case["op"] == "decode":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        hit = E * (1.0 - (1.0 - k / E) ** T)  # experts that T independent tokens are expected to reach
        per = 3 * H * I // 2 + 3 * H * I // BLOCK[case["fmt"]] * (4 if case["fmt"] == "nf4" else 1)
        b = hit * per + 4 * T * H + 8 * T * k + 4 * T * E
        f = 6 * T * k * H * I
        if case["router"]:
            b, f = b + 2 * E * H, f + 2 * T * E * H
        return {"bytes": int(b + (4 * E if case["bias"] else 0)), "flops": int(f)}
    if case["op"] == "step":
        M, I = case["T"] * case["k"], case["I"]
        n = M * (1.0 - case["drop"])
        # gate_up in, h and 8-bit gate_up out; 8-bit gate_up and dh in, d_gate_up out (and h once more)
        b = n * (4 * I + 2 * I + 66 * I // 32 + 66 * I // 32 + 2 * I + 4 * I + (2 * I if case["h_out"] else 0)) + 16 * M
        return {"bytes": int(b), "flops": int(n * I * 40)}
    if case["op"] == "combine_bwd":
        M, N = case["T"] * case["k"], case["N"]
        n = M * (1.0 - case["drop"])
        b = 2 * case["T"] * N + 2 * M * N + 4 * M  # dropped rows of dy are written as zeros
        if case["weighted"]:
            b += 4 * M
        if case["y"]:
            b += 2 * n * N + 8 * M
        return {"bytes": int(b), "flops": int(n * N * ((1 if case["weighted"] else 0) + (2 if case["y"] else 0)))}
    T, E, k = case["T"], case["E"], case["k"]
    return {"bytes": 12 * T * k + 4 * T * E, "flops": 4 * T * k}


# ---------------------------------------------------------------------------------------------------- exact values


def exact(case, seed):
    """The definitions in 64 bits, row by row or expert by expert."""
    s = prepare(case, seed)
    return {"decode": _decode_exact, "step": _step_exact, "combine_bwd": _combine_bwd_exact,
            "router_bwd": _router_bwd_exact}[case["op"]](s)


def _expert64(fmt, w, scales):
    """Dense fp64 weights of one expert, byte by byte through a 256-entry table of code pairs."""
    table = np.empty((256, 2))
    for b in range(256):
        table[b] = (NF4[b >> 4], NF4[b & 15]) if fmt == "nf4" else (E2M1[b & 15], E2M1[b >> 4])
    dense = torch.from_numpy(table).to(w.device)[w.int()].flatten(1)
    sc = scales.double() if fmt == "nf4" else torch.pow(torch.full_like(scales, 2, dtype=torch.float64),
                                                         scales.double() - 127)
    return dense * sc.repeat_interleave(BLOCK[fmt], dim=1)


def _decode_exact(s):
    T, k, I, H = s["T"], s["k"], s["I"], s["H"]
    x = s["x"].double()
    logits = torch.einsum("th,eh->te", x, s["router_w"].double()) if s["router"] else s["logits"].double()
    lg = logits.cpu().numpy()
    sc = lg if s["bias"] is None else lg + s["bias"].double().cpu().numpy()
    ids = np.stack([sorted(range(s["E"]), key=lambda e: (-sc[t, e], e))[:k] for t in range(T)])
    sel = np.take_along_axis(lg, ids, axis=1)
    p = np.exp(sel) / np.exp(sel).sum(axis=1, keepdims=True)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.reshape(-1).tolist())):
        ts, js = np.nonzero(ids == e)
        tt = torch.from_numpy(ts).cuda()
        gu = x[tt] @ _expert64(s["fmt"], s["w1"][e], s["s1"][e]).t()
        gate, up = gu[:, :I], gu[:, I:]
        y = (gate * torch.sigmoid(gate) * up) @ _expert64(s["fmt"], s["w2"][e], s["s2"][e]).t()
        out.index_add_(0, tt, y * torch.from_numpy(p[ts, js]).cuda()[:, None])
    return _decode_outputs(s, out, torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(p).cuda(), logits)


def _e4m3_64(a):
    """fp64 values to the nearest e4m3 value, ties to even (|a| below 448)."""
    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(a / step) * step


def _step_exact(s):
    I = s["I"]
    rows = torch.nonzero(s["s2f"] >= 0).flatten()
    M = s["gate_up"].shape[0]
    h = torch.zeros(M, I, dtype=torch.float64, device="cuda")
    h2, dgu = torch.zeros_like(h), torch.zeros(M, 2 * I, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["weights"].numel(), dtype=torch.float64, device="cuda")
    for part in rows.split(4096):
        gu = s["gate_up"][part].double()
        h[part] = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        blk = gu.reshape(len(part), -1, 32)
        top = blk.abs().amax(dim=2, keepdim=True)
        unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -126))) - 7.0).clamp(min=-127.0))
        q = (_e4m3_64(blk / unit) * unit).reshape(gu.shape)
        g, u = q.chunk(2, dim=1)
        sg = torch.sigmoid(g)
        dh, f = s["dh"][part].double(), s["s2f"][part].long()
        w = s["weights"].double().view(-1)[f].unsqueeze(1)
        dgu[part] = torch.cat((w * dh * u * (sg + g * sg * (1 - sg)), w * dh * g * sg), dim=1)
        h2[part] = g * sg * u
        dw[f] = (dh * h2[part]).sum(dim=1)
    out = {"h": h, "d_gate_up": dgu, "d_weights": dw.view(s["weights"].shape)}
    if s["h_out"]:
        out["h2"] = h2
    return out


def _combine_bwd_exact(s):
    k, N = s["k"], s["N"]
    dy = torch.zeros(s["T"] * k, N, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["T"], k, dtype=torch.float64, device="cuda")
    for j in range(k):  # slot by slot of every token
        r = s["f2s"].view(-1, k)[:, j].long()
        t = torch.nonzero(r >= 0).flatten()
        d = s["dout"][t].double()
        dy[r[t]] = d if s["weights"] is None else d * s["weights"][t, j].double()[:, None]
        if s["y"] is not None:
            dw[t, j] = torch.einsum("tn,tn->t", d, s["y"][r[t]].double())
    return {"dy": dy} if s["y"] is None else {"dy": dy, "d_weights": dw}


def _router_bwd_exact(s):
    p, dw = s["wts"].double(), s["d_weights"].double()
    jac = torch.diag_embed(p) - p.unsqueeze(2) * p.unsqueeze(1)
    d = torch.bmm(jac, dw.unsqueeze(2)).squeeze(2)
    out = torch.zeros(s["T"], s["E"], dtype=torch.float64, device="cuda")
    out[torch.arange(s["T"], device="cuda")[:, None], s["ids"].long()] = d
    return out
