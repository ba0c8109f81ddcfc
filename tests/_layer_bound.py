"""The whole-layer decode's error bound, from the roundings that its header states and nothing else:

    x             exact, but values below 2^-28 of the token's largest |x|: within 2^-39 of that;
    NF4 codes     rounded to fp16 (the error of each of the 16 is computed here); MXFP4 codes exact;
    p * h         rounded to 11 bits (half a step: 2^-11), within 2^-39 of the pair's largest below 2^-28 of it;
    sums, scales  fp32: n terms lose at most n * 2^-24 of the sum of their absolute values;
    activation    __expf 2 + 1.16 |g| units, the fast division 2, three more operations: (8 + 1.2 |g|) 2^-23;
    p             expf, k terms and a division: (k + 16) 2^-24, and its product with h;
    out           rounded to bf16 once: 2^-8.

An error of the gate moves h by at most 1.1 |u| times as much (the largest slope of silu is 1.0999)."""
from __future__ import annotations

import numpy as np

from tests import _layer_ref as ref

CODE_ERROR = np.abs(ref.NF4.astype(np.float16).astype(np.float64) - ref.NF4)


def code_errors(fmt, w, scales):
    """|weight as the kernel has it - weight|, fp64 [N, K]."""
    if fmt == "mxfp4":
        return np.zeros((w.shape[0], 2 * w.shape[1]))
    v = np.stack([CODE_ERROR[w >> 4], CODE_ERROR[w & 15]], -1).reshape(w.shape[0], -1)
    return v * np.repeat(np.abs(np.asarray(scales, np.float64)), 64, axis=1)


def small(v):
    """Absolute error of v as fp16 scaled by its largest: 0 or, below 2^-28 of it, 2^-39 of it."""
    top = np.abs(v).max()
    return np.where(np.abs(v) < 2.0 ** -28 * top, 2.0 ** -39 * top, 0.0)


def layer(fmt, x, ids, p, w1, s1, w2, s2, round_h=None):
    """out [T, H] in fp64 and the bound, element by element.  round_h: p * h goes through it before the down projection."""
    x = np.asarray(x, np.float64)
    T, k = ids.shape
    H, I = x.shape[1], w1.shape[1] // 2
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for e in sorted(set(ids.reshape(-1).tolist())):
        W1, W2 = ref.dequant(fmt, w1[e], s1[e]), ref.dequant(fmt, w2[e], s2[e])
        D1, D2 = code_errors(fmt, w1[e], s1[e]), code_errors(fmt, w2[e], s2[e])
        A1, A2 = np.abs(W1), np.abs(W2)
        for t, j in zip(*np.nonzero(ids == e)):
            ax = np.abs(x[t]) + small(x[t])
            gu = W1 @ x[t]
            e1 = D1 @ ax + A1 @ small(x[t]) + (H + 8) * 2.0 ** -24 * ((A1 + D1) @ ax)
            g, up = gu[:I], gu[I:]
            act = g * ref.sigmoid(g)
            ph = p[t, j] * act * up
            eh = 1.1 * np.abs(up) * e1[:I] + np.abs(act) * e1[I:] + 1.1 * e1[:I] * e1[I:]
            eh = p[t, j] * eh + np.abs(ph) * ((8 + 1.2 * np.abs(g)) * 2.0 ** -23 + (k + 20) * 2.0 ** -24)
            size = np.abs(ph) + eh
            eh = eh + size * 2.0 ** -11 + np.where(size < 2.0 ** -27 * size.max(), 2.0 ** -39 * size.max(), 0.0)
            out[t] += W2 @ (ph if round_h is None else round_h(ph))
            err[t] += (A2 + D2) @ eh + D2 @ np.abs(ph) + (k * I + 64) * 2.0 ** -24 * ((A2 + D2) @ size)
    return out, err * (1 + 2.0 ** -8) + np.abs(out) * 2.0 ** -8 + 2.0 ** -133


def rms_limit(fmt, want, bf16):
    """Largest rms error over rms value, for some ten thousand outputs: that of rounding `want` itself to bf16 (bf16: a
    function doing so), and independently of it the roundings in front: p * h, evenly spread in half a step of 2^-11
    (a third of its square); and for NF4 every code, at most 2^-11 of it, in the down projection, in up, and in gate,
    where silu carries a relative error of g on at most 1.5 times in the mean.  3% for the sample."""
    before = 2.0 ** -22 * (1 / 3 + (0 if fmt == "mxfp4" else 1 + 1 + 1.5 ** 2))
    return 1.03 * np.sqrt(((bf16(want) - want) ** 2).mean() / (want ** 2).mean() + before)


def rms(got, want):
    return np.sqrt(((got - want) ** 2).mean() / (want ** 2).mean())
