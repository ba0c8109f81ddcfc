"""Plain 64-bit definitions of the whole-layer and training calls, on the CPU (no library code)."""
from __future__ import annotations

import numpy as np
import torch

NF4 = np.array([-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
                -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
                0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941, 0.7229568362236023,
                1.0])
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def dequant(fmt, w, scales):
    """Packed rows uint8 [N, K/2] -> fp64 [N, K]."""
    w = np.asarray(w)
    hi, lo = w >> 4, w & 15
    if fmt == "nf4":
        v = np.stack([NF4[hi], NF4[lo]], -1).reshape(w.shape[0], -1)
        return v * np.repeat(np.asarray(scales, np.float64), 64, axis=1)
    v = np.stack([E2M1[lo], E2M1[hi]], -1).reshape(w.shape[0], -1)
    s = np.asarray(scales).astype(np.int64)
    return v * np.repeat(np.where(s == 255, np.nan, np.ldexp(1.0, s - 127)), 32, axis=1)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def topk(logits, bias, k):
    """Descending by logit + bias in fp32, ties to the lower index, NaN last; softmax of the raw logits."""
    lg = np.asarray(logits, np.float32)
    sc = lg if bias is None else lg + np.asarray(bias, np.float32)[None]
    ids = np.empty((lg.shape[0], k), np.int32)
    for t in range(lg.shape[0]):
        order = sorted(range(lg.shape[1]), key=lambda e: (bool(np.isnan(sc[t, e])), 0.0 if np.isnan(sc[t, e]) else -sc[t, e], e))
        ids[t] = order[:k]
    sel = np.take_along_axis(lg.astype(np.float64), ids, 1)
    with np.errstate(invalid="ignore"):
        p = np.exp(sel - sel.max(1, keepdims=True))
        return ids, p / p.sum(1, keepdims=True)


def layer(fmt, x, ids, p, w1, s1, w2, s2):
    """out [T, H] in fp64 and a bound on the kernel's error, element by element.

    The bound counts roundings to bf16 (u = 2^-8, half a step): the output once, w * h once, and for NF4 every code of
    both projections once; MXFP4 weights are exact.  An error e of a weight moves a product by e |w x|; an error of the
    gate moves h by at most 1.1 |u| (the largest slope of silu is 1.0999).  fp32 sums of n terms: n * 2^-24 of the sum
    of absolute terms, plus 2^-20 for the exponential, the division and the multiplications of the activation."""
    x = np.asarray(x, np.float64)
    T, k = ids.shape
    H, I = x.shape[1], w1.shape[1] // 2
    u = 2.0 ** -8
    code = u if fmt == "nf4" else 0.0
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for e in sorted(set(ids.reshape(-1).tolist())):
        W1, W2 = dequant(fmt, w1[e], s1[e]), dequant(fmt, w2[e], s2[e])
        A1, A2 = np.abs(W1), np.abs(W2)
        for t, j in zip(*np.nonzero(ids == e)):
            gu, agu = W1 @ x[t], A1 @ np.abs(x[t])
            g, up = gu[:I], gu[I:]
            e1 = agu * (code + H * 2.0 ** -24)
            act = g * sigmoid(g)
            h = act * up
            eh = 1.1 * np.abs(up) * e1[:I] + np.abs(act) * e1[I:] + 1.1 * e1[:I] * e1[I:] + np.abs(h) * 2.0 ** -20
            out[t] += p[t, j] * (W2 @ h)
            eh = eh * (1 + u) + np.abs(h) * u
            err[t] += p[t, j] * (A2 @ eh * (1 + code) + (A2 @ np.abs(h)) * (code + (k * I + 64) * 2.0 ** -24 + 2.0 ** -20))
    return out, err * (1 + u) + np.abs(out) * u + 2.0 ** -133


def e4m3(a):
    """Nearest e4m3 value of |a| <= 448, ties to even."""
    a = np.asarray(a, np.float64)
    mag = np.maximum(np.abs(a), 2.0 ** -6)
    step = np.exp2(np.floor(np.log2(mag)) - 3)
    return np.round(a / step) * step


def ckpt8(v):
    """bf16 values [M, C] (fp64) -> the values their 8-bit checkpoint stands for, and the scale bytes."""
    b = np.asarray(v, np.float64).reshape(v.shape[0], -1, 32)
    fin = np.isfinite(b)
    top = np.where(fin, np.abs(b), 0.0).max(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        X = np.where(top > 0, np.floor(np.log2(np.maximum(top, 1e-300))) - 7, -127)
    X = np.maximum(X, -127)
    q = np.where(fin, e4m3(np.where(fin, b, 0.0) / np.exp2(X)) * np.exp2(X), np.nan)
    return q.reshape(v.shape), (X[..., 0] + 127).astype(np.uint8)


def decode_ckpt(codes, scales):
    """codes uint8 [M, C], scales uint8 [M, C/32] -> fp64 values, from the e4m3 definition."""
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    v = np.where((c & 127) == 127, np.nan, np.where(c & 128, -v, v))
    return v * np.repeat(np.exp2(np.asarray(scales).astype(np.float64) - 127), 32, axis=1)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.dtype == torch.bfloat16 else \
        t.detach().cpu().numpy().astype(np.float64)
