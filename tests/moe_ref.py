"""Plain 64-bit implementations of the mixture-of-experts operators for the
tests: one token, pair or row at a time, numpy float64, from the definitions
in include/hocf.h."""

import math

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def scores(x, score):
    """(scores, on) of one row of logits in 64 bits; -inf and NaN are switched off."""
    x = np.asarray(x, np.float64)
    on = x > -np.inf
    s = np.zeros(len(x))
    if not on.any():
        return s, on
    if score == SOFTMAX:
        top = x[on].max()
        with np.errstate(invalid="ignore"):
            s[on] = np.where(x[on] == top, 1.0, np.exp(x[on] - top))
        s /= s.sum()
    else:
        with np.errstate(over="ignore"):
            s[on] = 1.0 / (1.0 + np.exp(-x[on]))
    return s, on


def route(logits, topk, bias=None, score=SOFTMAX, n_group=1, topk_group=1, group_top=1, renorm=False, scale=1.0):
    T, E = logits.shape
    experts = np.full((T, topk), -1, np.int32)
    weights = np.zeros((T, topk))
    for t in range(T):
        s, on = scores(logits[t], score)
        v = np.where(on, s + (0.0 if bias is None else bias.astype(np.float64)), -np.inf)
        size = E // n_group
        if n_group > 1:
            of = []
            for g in range(n_group):
                best = sorted(v[g * size:(g + 1) * size], reverse=True)[:group_top]
                best = [b for b in best if b > -np.inf]
                of.append(sum(best) if best else -np.inf)
            kept = sorted(range(n_group), key=lambda g: (-of[g], g))[:topk_group]
            v = np.array([v[e] if e // size in kept else -np.inf for e in range(E)])
        order = [e for e in sorted(range(E), key=lambda e: (-v[e], e)) if v[e] > -np.inf][:topk]
        experts[t, :len(order)] = order
        total = sum(s[e] for e in order) if renorm else 1.0
        for j, e in enumerate(order):
            weights[t, j] = scale * s[e] / total if total else 0.0
    counts = np.bincount(experts[experts >= 0], minlength=E)[:E]
    return experts, weights, counts


def weights_of(logits, experts, score, renorm, scale):
    """The weights of given experts (the choice held fixed), for differences."""
    out = np.zeros(experts.shape)
    for t in range(len(logits)):
        s, _ = scores(logits[t], score)
        w = np.array([s[e] if e >= 0 else 0.0 for e in experts[t]])
        out[t] = scale * (w / w.sum() if renorm and w.sum() else w)
    return out


def route_bwd(logits, experts, dweights, score, renorm, scale):
    """(dlogits, size): the gradient by the chain rule, and the sum of the magnitudes that it is a sum of."""
    T, E = logits.shape
    d = np.zeros((T, E))
    size = np.zeros((T, E))
    for t in range(T):
        s, on = scores(logits[t], score)
        e = [(j, k) for j, k in enumerate(experts[t]) if 0 <= k < E and on[k]]
        g = {j: float(dweights[t, j]) * scale for j, _ in e}
        ds = np.zeros(E)           # gradient of the scores
        mag = np.zeros(E)
        total = sum(s[k] for _, k in e)
        for j, k in e:
            if renorm:
                if total:
                    ds[k] += g[j] / total - sum(g[i] * s[m] for i, m in e) / total ** 2
                    mag[k] += abs(g[j]) / total + sum(abs(g[i]) * s[m] for i, m in e) / total ** 2
            else:
                ds[k] += g[j]
                mag[k] += abs(g[j])
        if score == SOFTMAX:
            d[t] = s * (ds - (ds * s).sum())
            size[t] = s * (mag + (mag * s).sum())
        else:
            d[t] = ds * s * (1 - s)
            size[t] = mag * s * (1 - s)
    return d, size


def slots(experts, bins, per_bin, cap):
    index = np.full(experts.shape, -1, np.int32)
    pair = np.full(bins * cap, -1, np.int32)
    counts = np.zeros(bins, np.int64)
    flat = index.reshape(-1)
    for i, e in enumerate(experts.reshape(-1)):
        if 0 <= e < bins * per_bin:
            b = e // per_bin
            if counts[b] < cap:
                flat[i] = b * cap + counts[b]
                pair[flat[i]] = i
            counts[b] += 1
    return index, pair, counts


def combine(rows, weights, index, add=None):
    T, topk = weights.shape
    out = np.zeros((T, rows.shape[1])) if add is None else add.astype(np.float64).copy()
    size = np.abs(out)
    for t in range(T):
        for j in range(topk):
            r = t * topk + j if index is None else index[t, j]
            if r >= 0:
                out[t] += float(weights[t, j]) * rows[r].astype(np.float64)
                size[t] += abs(float(weights[t, j])) * np.abs(rows[r].astype(np.float64))
    return out, size


def combine_bwd(rows, weights, dout, index):
    T, topk = weights.shape
    drows = np.zeros(rows.shape)
    dw = np.zeros((T, topk))
    size = np.zeros((T, topk))
    for t in range(T):
        for j in range(topk):
            r = t * topk + j if index is None else index[t, j]
            if r >= 0:
                drows[r] = float(weights[t, j]) * dout[t].astype(np.float64)
                q = rows[r].astype(np.float64) * dout[t].astype(np.float64)
                dw[t, j], size[t, j] = q.sum(), np.abs(q).sum()
    return drows, dw, size


def w4(x, codes, scales, zeros, experts, e0, rows_per_x, group):
    """out[r] = x[r // rows_per_x] . W[experts[r] - e0]; (out, sum of magnitudes incl. the offset of 24)."""
    E, K, N = codes.shape
    R = len(x) * rows_per_x if experts is None else len(experts)
    out, size = np.zeros((R, N)), np.zeros((R, N))
    of = np.arange(K) // group
    for r in range(R):
        e = 0 if experts is None else int(experts[r]) - e0
        if not 0 <= e < E:
            continue
        s = scales[e][of].astype(np.float64)
        z = 8.0 if zeros is None else zeros[e][of].astype(np.float64)
        xr = x[r // rows_per_x].astype(np.float64)
        out[r] = xr @ (s * (codes[e] - z))
        size[r] = np.abs(xr) @ (np.abs(s) * (np.abs(z) + 31.0))
    return out, size


def rel_steps(n):
    """n half steps of binary32."""
    return n * math.ldexp(1.0, -24)
