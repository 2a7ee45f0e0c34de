"""The operators of include/wd_step.h and the rotation of include/wd_kv.h in plain numpy, 64 bits.

Written from the definitions in the headers, and sharing no code with the library.
"""
import numpy as np

E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def e4m3_values(codes):
    c = np.asarray(codes, np.uint8)
    return np.where((c & 127) == 127, np.nan, np.append(E4M3, np.nan)[c & 127]) * np.where(c >= 128, -1.0, 1.0)


def e8m0_values(scales):
    return np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))


def rms_norm(x, weight, residual, eps):
    """(y, r), float64."""
    r = x + (0.0 if residual is None else residual)
    with np.errstate(invalid="ignore", over="ignore"):
        y = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return y * (1.0 if weight is None else weight), r


def route(x, K, scores, bias, groups, top_groups, group_best, renormalise, scale):
    """ids [T, K] and weights, float64, one token after the other."""
    T, E = x.shape
    size = E // groups
    ids, weights = np.zeros((T, K), np.int64), np.zeros((T, K))
    for t in range(T):
        l = np.where(np.isnan(x[t]), -np.inf, x[t])
        there = l > -np.inf
        score = np.zeros(E)
        with np.errstate(over="ignore"):
            if scores == "sigmoid":
                score[there] = 1 / (1 + np.exp(-l[there]))
            elif there.any():
                top = l.max()
                e = np.where(l == top, 1.0, np.exp(np.where(there, l, 0) - (top if np.isfinite(top) else 0)))
                if np.isinf(top):
                    e = (l == top).astype(float)
                e[~there] = 0
                score = e / e.sum()
        key = score + bias if bias is not None else score
        key = np.where(there & ~np.isnan(key), key, -np.inf)
        by = key if bias is not None else l  # ordered as the scores are, and exact
        if groups > 1 and top_groups < groups:
            value = np.zeros(groups)
            for g in range(groups):
                if group_best == 1:
                    value[g] = by[g * size:(g + 1) * size].max()
                else:
                    a = np.sort(key[g * size:(g + 1) * size])[::-1][:2]
                    value[g] = a[0] + a[1] if len(a) == 2 and a[1] > -np.inf else a[0]
            chosen = np.argsort(-value, kind="stable")[:top_groups]
            open_ = np.isin(np.arange(E) // size, chosen)
        else:
            open_ = np.ones(E, bool)
        order = sorted(np.flatnonzero(open_), key=lambda e: (-by[e], e))[:K]
        ids[t] = order
        w = score[order]
        if renormalise:
            if scores == "sigmoid":  # in logarithms, where far negative logits leave 64 bits too
                lo = np.array([-np.logaddexp(0, -l[e]) if there[e] else -np.inf for e in order])
            else:
                lo = np.array([l[e] if there[e] else -np.inf for e in order])
            top = lo.max()
            if top == -np.inf:
                w = np.zeros(K)
            else:
                w = np.array([1.0 if v == top else np.exp(v - top) if np.isfinite(top) else 0.0 for v in lo])
                w = w / w.sum()
        weights[t] = w * scale
    return ids, weights


def adjust_logits(x, history=None, lengths=None, prompt_lengths=None, seqs=None, repetition=None, presence=None,
                  frequency=None, bias=None, temperature=None, mask=None):
    """(want, the magnitudes that its sums are made of), float64 [B, V]."""
    B, V = x.shape
    want, mag = x.copy(), np.abs(x)
    with np.errstate(invalid="ignore", divide="ignore"):
        for b in range(B):
            l, m = want[b], mag[b]
            slot = b if seqs is None else int(seqs[b])
            if history is not None and 0 <= slot < history.shape[0]:
                n = min(max(int(lengths[slot]), 0), history.shape[1])
                p = 0 if prompt_lengths is None else min(max(int(prompt_lengths[slot]), 0), n)
                t = history[slot, :n]
                fine = (t >= 0) & (t < V)
                rep = 1.0 if repetition is None else repetition[b]
                for v in np.unique(t[fine]):
                    l[v] = l[v] / rep if l[v] > 0 else l[v] * rep
                    m[v] = np.abs(l[v])
                answer, times = np.unique(t[p:][fine[p:]], return_counts=True)
                f = 0.0 if frequency is None else frequency[b]
                pr = 0.0 if presence is None else presence[b]
                l[answer] -= times * f + pr
                m[answer] += np.abs(times * f) + np.abs(pr)
            if bias is not None:
                start, ids, values = bias
                lo, hi = int(start[b]), int(start[b + 1])
                if 0 <= lo <= hi <= len(ids):
                    for v, z in zip(ids[lo:hi], values[lo:hi]):
                        if 0 <= v < V:
                            l[v] += float(z)
                            m[v] += abs(float(z))
            if temperature is not None and temperature[b] > 0:
                l /= temperature[b]
                m /= temperature[b]
            if mask is not None:
                words = mask[b].astype(np.uint32)
                bits = (words[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
                l[bits == 0] = -np.inf
    return want, mag


def rotate(x, cos_sin, pos, paired):
    """x float32 [T, heads, D] turned by FP32 products and sums, rounded one by one."""
    R = cos_sin.shape[1]
    y = x.astype(np.float32).copy()
    for t in range(x.shape[0]):
        c, s = cos_sin[pos[t], :R // 2].astype(np.float32), cos_sin[pos[t], R // 2:].astype(np.float32)
        i1, i2 = (np.arange(0, R, 2), np.arange(1, R, 2)) if paired else (np.arange(R // 2), np.arange(R // 2, R))
        a, b = x[t][:, i1].astype(np.float32), x[t][:, i2].astype(np.float32)
        with np.errstate(invalid="ignore", over="ignore"):
            y[t][:, i1] = a * c - b * s
            y[t][:, i2] = b * c + a * s
    return y
