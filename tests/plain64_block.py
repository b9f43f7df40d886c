"""Plain forms in 64 bits of the norms around a block, their gradient and the whole layer for a few tokens, with bounds
on what fp32 arithmetic may be off by. numpy, from the formulas; nothing here comes from the package.

Bounds. u = 2^-24 is half a step of fp32. A row's sum takes at most 32 terms in a thread's chain, 5 steps of a
butterfly, and 5 more over at most 32 warps: at most 42 roundings, 64 with room for the terms' own products. So a mean
of squares (terms of one sign) is off by at most 64 u of itself, its inverse root by 32 u and the 2 u of the root's own
rounding: ROOT = 40 u. Every other step is a product or a fused sum, counted one u each."""
import numpy as np

U = 2.0 ** -24
ROOT = 40 * U


def inv_rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def gate_of(gate, kind, T):
    if kind == "none":
        return np.ones((T, 1))
    g = gate.astype(np.float64)
    return g[:, None] if kind == "token" else g[None, :]


def forward(y, dy, residual, w_post, w_pre, gate, kind, scale, eps):
    """r, n and the bounds on their errors before the final rounding. dy: the bound on y's own error (or 0)."""
    f = gate_of(gate, kind, residual.shape[0]) * scale
    if y is None:
        r, dr = residual, np.zeros_like(residual)
    else:
        b, db = y, dy + np.zeros_like(y)
        if w_post is not None:
            s = inv_rms(y, eps)
            # the root follows y's errors by their share of its norm
            moved = np.sqrt((db * db).sum(1, keepdims=True)) / np.sqrt((y * y).sum(1, keepdims=True) + y.shape[1] * eps)
            b = y * s * w_post
            db = np.abs(s * w_post) * db + np.abs(b) * (ROOT + moved)
        r = residual + f * b
        dr = np.abs(f) * (db + 4 * U * np.abs(b)) + U * np.abs(r)
    if w_pre is None:
        return r, dr, None, None
    s = inv_rms(r, eps)
    n = r * s * w_pre
    moved = np.sqrt((dr * dr).sum(1, keepdims=True)) / np.sqrt((r * r).sum(1, keepdims=True) + r.shape[1] * eps)
    return r, dr, n, np.abs(s * w_pre) * dr + np.abs(n) * (ROOT + moved + 2 * U)


def backward(y, r, d_r, d_n, w_post, w_pre, gate, kind, scale, eps):
    """The gradients by the formulas, each with a bound: (value, bound) by name. m* are sums of magnitudes: every
    result is linear in the magnitudes that it is formed from, and each of its at most 4 sums and roots adds 64 u of
    them, each of its at most 20 other steps one u: 300 u covers all; a sum over T tokens adds T + 100."""
    T, H = r.shape if r is not None else d_r.shape
    out = {}
    D = np.zeros((T, H)) if d_r is None else d_r
    mD = np.abs(D)
    if w_pre is not None:
        s = inv_rms(r, eps)
        rh, v = r * s, w_pre * d_n
        D = D + s * (v - rh * (rh * v).mean(1, keepdims=True))
        mD = mD + s * (np.abs(v) + np.abs(rh) * np.abs(rh * v).mean(1, keepdims=True))
        m = np.abs(d_n * rh).sum(0)
        out["d_w_pre"] = ((d_n * rh).sum(0), (T + 200) * U * m)
    out["d_residual"] = (D, 300 * U * mD)
    if y is None:
        return out
    g = gate_of(gate, kind, T)
    c, mc = scale * g * D, np.abs(scale * g) * mD
    b = y
    if w_post is None:
        out["d_y"] = (c, 300 * U * mc)
    else:
        s = inv_rms(y, eps)
        yh, v, mv = y * s, w_post * c, np.abs(w_post) * mc
        b = yh * w_post
        out["d_y"] = (s * (v - yh * (yh * v).mean(1, keepdims=True)),
                      300 * U * s * (mv + np.abs(yh) * (np.abs(yh) * mv).mean(1, keepdims=True)))
        out["d_w_post"] = ((c * yh).sum(0), (T + 400) * U * (mc * np.abs(yh)).sum(0))
    if kind == "channel":
        out["d_gate"] = (scale * (D * b).sum(0), (T + 400) * U * abs(scale) * (mD * np.abs(b)).sum(0))
    if kind == "token":
        out["d_gate"] = (scale * (D * b).sum(1), 400 * U * abs(scale) * (mD * np.abs(b)).sum(1))
    return out


def combine(y, idx, w, slot):
    """The weighted sum of the experts' rows, and the bound of its fp32 form: a rounding a choice."""
    T, k = idx.shape
    out, mag = np.zeros((T, y.shape[2])), np.zeros((T, y.shape[2]))
    for t in range(T):
        for j in range(k):
            if slot[t, j] >= 0:
                v = w[t, j] * y[idx[t, j], slot[t, j]]
                out[t] += v
                mag[t] += np.abs(v)
    return out, k * U * mag


def bf16(a):
    """The bf16 values that float64 values round to (through fp32, which moves a value by 2^-24 of it at most)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).float().to(torch.bfloat16).double().numpy()


def mlp(x, up, down, inner, half=False, up_mag=None, down_mag=None):
    """One expert's MLP of rows x in float64, up [2 inner][H], down [H][inner], with h rounded to bf16 as the layer's
    definition has it; and a bound on what the fp32 sums may move the result by. half (weights of 8 and 4 bits): the inputs
    of both products are fp16 behind a power of two for each row, h not rounded before: every h may be off by 2^-11 of it
    (half a step of fp16), and every input by 2^-35 of its row's largest (half of fp16's lowest step, 2^-25, where the
    largest is 2^14 or more, and 16 times that where inputs are divided by 16).

    A product of K inputs: an MMA step of 16 rounds its sum and its add into the accumulator (2), at most K/16 steps; a
    group's sum is scaled and added (2 for each of K/32 groups at most); 8 partial sums are joined, and at most 8 blocks':
    (K/8 + K/16 + 24) u of the sum of magnitudes =: B. up_mag, down_mag (4-bit weights): the group's scale times 1040, the
    largest operand that stands for a code; within a group of at most 128 inputs the sum is of these, from a start that is a
    rounded sum itself: 16 roundings of 8 MMA steps and 36 of the start, 52 u of their magnitudes more. silu moves by at most
    1.1 of its argument's error and is formed in 4 roundings more, 2^-21 in all. Where that reach crosses a rounding border
    of bf16, h may be the neighbour: its reach is the difference of the rounded ends. Down, h's reach goes through the
    magnitudes, and the product's own B is added."""
    def product(v, w, mag):
        K = w.shape[1]
        B = (K / 8 + K / 16 + 24) * U * (np.abs(v) @ np.abs(w).T)
        if half:
            B = B + 2.0 ** -35 * np.abs(v).max(1, keepdims=True) * np.abs(w).sum(1)
        if mag is not None:
            B = B + 52 * U * (np.abs(v) @ mag.T)
        return v @ w.T, B
    r, B = product(x, up, up_mag)
    g, u, Bg, Bu = r[:, :inner], r[:, inner:], B[:, :inner], B[:, inner:]
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    h = s * u
    reach = 1.1 * Bg * np.abs(u) + np.abs(s) * Bu + Bg * Bu + 2.0 ** -21 * np.abs(h)
    if half:
        reach, hr = reach + 2.0 ** -11 * np.abs(h), h
    else:
        hr = bf16(h)
        reach = np.maximum(np.abs(bf16(h + reach) - hr), np.abs(bf16(h - reach) - hr))
    out, Bo = product(hr, down, down_mag)
    return out, Bo + reach @ np.abs(down).T
