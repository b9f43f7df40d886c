"""Plain forms in 64 bits of the gated route, the gradients and the 4-bit expert products, for the tests: numpy,
from the formulas, with loops where they are the plainest. Nothing here comes from the package."""
import numpy as np

MASK_LOGIT = -(2.0 - 2.0 ** -7) * 2.0 ** 127          # the lowest finite bf16


def bf16_round(a):
    """float64/float32 -> the bf16 value as float32, round to nearest even (from the fp32 value)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def gate(logits, bias, k, G=1, top_g=1, top2=False, sigmoid=True, renorm=True, scale=1.0):
    """(idx [T][k], ok [T][k], w [T][k], margin [T]): the choice with its weights. margin: how near the token's
    choice came to another one, the least gap between keys (or group scores) whose order matters."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    per = E // G
    idx, ok, w = np.zeros((T, k), np.int32), np.zeros((T, k), bool), np.zeros((T, k))
    margin = np.full(T, np.inf)
    for t in range(T):
        open_ = l[t] > MASK_LOGIT                                   # False for NaN and -inf
        if bias is not None:
            open_ &= np.asarray(bias, np.float64) > -np.inf         # False for NaN too
        s = scores(l[t], sigmoid)
        key = np.where(open_, l[t] if bias is None else s + bias, -np.inf)
        by = s if bias is None else s + bias
        live = np.ones(E, bool)
        if G > 1:
            score = np.zeros(G)
            for g in range(G):
                m = slice(g * per, (g + 1) * per)
                if top2:
                    b = sorted(by[m][open_[m]], reverse=True)
                    score[g] = b[0] + b[1] if len(b) >= 2 else -np.inf
                else:
                    score[g] = key[m].max()
            order = sorted(range(G), key=lambda g: (-score[g], g))
            if top_g < G and np.isfinite(score[order[top_g]]):
                gap = score[order[top_g - 1]] - score[order[top_g]]
                margin[t] = min(margin[t], gap if gap > 0 else np.inf)
            live[:] = False
            for g in order[:top_g]:
                live[g * per:(g + 1) * per] = True
        real = sorted(np.nonzero(live & open_)[0], key=lambda e: (-key[e], e))
        rest = [e for e in range(E) if not (live[e] and open_[e])]
        for a, b in zip(real[:k], real[1:k + 1]):
            if np.isfinite(key[a]) and np.isfinite(key[b]) and key[a] > key[b]:
                margin[t] = min(margin[t], key[a] - key[b])
        pick = (real + rest)[:k]
        n = min(k, len(real))
        idx[t], ok[t, :n] = pick, True
        w[t, :n] = chosen_weights(l[t][pick[:n]], s[pick[:n]], sigmoid, renorm) * scale
    return idx, ok, w, margin


def chosen_weights(l, s, sigmoid, renorm):
    """The weights of the chosen logits l with scores s, before the scale; quotients by their logarithms, which do
    not underflow."""
    if not renorm or len(l) == 0:
        return s
    if not sigmoid:
        return scores(l, False)
    log_s = -np.logaddexp(0.0, -l)
    c = np.exp(log_s - log_s.max())
    return c / c.sum()


def scores(l, sigmoid):
    if sigmoid:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    open_ = l > MASK_LOGIT
    if not open_.any():
        return np.zeros_like(l)
    top = l[open_].max()
    e = np.zeros_like(l)
    with np.errstate(invalid="ignore"):
        e[open_] = np.where(l[open_] == top, 1.0, np.exp(l[open_] - top))
    return e / e.sum()


def count(idx, ok, E, R, C):
    """counts, offsets, slot, rank_counts, dropped of the pairs, token by token."""
    counts, slot = np.zeros(E, np.int32), np.full(idx.shape, -1, np.int32)
    for t in range(idx.shape[0]):
        for j in range(idx.shape[1]):
            if ok[t, j]:
                e = idx[t, j]
                if counts[e] < C:
                    slot[t, j] = counts[e]
                counts[e] += 1
    kept = np.minimum(counts, C)
    return {"counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), "slot": slot,
            "rank_counts": kept.reshape(R, -1).sum(1).astype(np.int32), "dropped": int((counts - kept).sum())}


def weights_of(l, idx, ok, sigmoid, renorm, scale):
    """topk_w of one token as a function of its logits, the choice held fixed."""
    s = scores(l, sigmoid)[idx] * ok
    return (s / s.sum() if renorm else s) * scale


def gate_backward(logits, idx, ok, d_w, sigmoid, renorm, scale):
    """d_logits, and a bound on the sum of the magnitudes that each element is formed from."""
    l = np.asarray(logits, np.float64)
    d, mag = np.zeros_like(l), np.zeros_like(l)
    for t in range(l.shape[0]):
        i, v = idx[t][ok[t]], d_w[t][ok[t]].astype(np.float64)
        if len(i) == 0:
            continue
        s = scores(l[t], sigmoid)
        c = chosen_weights(l[t][i], s[i], sigmoid, renorm)
        dot, adot = (c * v).sum(), np.abs(c * v).sum()
        if sigmoid:
            inner = v - dot if renorm else v
            one_less = 1.0 / (1.0 + np.exp(np.minimum(l[t][i], 700)))
            d[t, i] = scale * c * one_less * inner
            mag[t, i] = abs(scale) * c * one_less * (np.abs(v) + adot)
        elif renorm:
            d[t, i] = scale * c * (v - dot)
            mag[t, i] = abs(scale) * c * (np.abs(v) + adot)
        else:
            full = np.zeros(l.shape[1])
            full[i] = v
            d[t] = scale * s * (full - dot)
            mag[t] = abs(scale) * s * (np.abs(full) + adot)
    return d, mag


def w4_codes(w_q, K):
    """4-bit codes [..., K] of packed bytes [..., K/2], by the layout's words."""
    word = np.ascontiguousarray(w_q).view("<u4")
    out = np.zeros(w_q.shape[:-1] + (K,), np.int64)
    for i in range(K):
        b, r = divmod(i, 128)
        j, r = divmod(r, 32)
        t, r = divmod(r, 8)
        out[..., i] = (word[..., 16 * b + 4 * t + j] >> (4 * (r // 2) + 16 * (r % 2))) & 15
    return out


def w4_rows(x, codes, scale, group):
    """r [c][M] = sum_i x (q - 8) scale, and the sum of magnitudes, for one expert in float64."""
    w = (codes - 8.0) * np.repeat(scale.astype(np.float64), group, axis=1)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))
