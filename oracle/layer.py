"""Reference of the operators around the grouped GEMMs, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The general router (scores, balance bias, groups, top-k, renormalised
weights), its gradient, the block alignment of given ids with a window of
local experts, and the dense int8 product with a scale per token and per
channel.  Each follows its definition token by token or element by element.
"""

import numpy as np

SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


def _softmax(v):
    """exp(v) / sum exp(v); all zero where nothing is above -inf."""
    m = np.max(v) if not np.isnan(v).any() else np.nan
    if m == -np.inf:
        return np.zeros_like(v)
    with np.errstate(invalid="ignore"):
        e = np.exp(v - m)
        return e / e.sum()


def _sigmoid(v):
    e = np.exp(-np.abs(v))                   # does not overflow
    return np.where(np.asarray(v) < 0, e, 1.0) / (1.0 + e)


def _to_38_bits(v):
    """v with 38 bits behind its leading one: sums that are equal in exact
    arithmetic (sigmoid(x) + sigmoid(-x) = 1) are equal here too, where their
    float64 evaluations differ in the last bit."""
    if not np.isfinite(v):
        return v
    m, e = np.frexp(v)
    return float(np.ldexp(np.rint(np.ldexp(m, 39)), int(e) - 39))


def _ranked(values, indices):
    """indices by value: NaN first, then the larger value, on equal values the
    lower index."""
    nan = [i for i in indices if np.isnan(values[i])]
    rest = sorted((i for i in indices if not np.isnan(values[i])), key=lambda i: (-values[i], i))
    return nan + rest


def route_general(logits, bias, top_k, score=SOFTMAX, n_group=1, topk_group=1,
                  group_rule=GROUP_MAX, renormalize=True, scale=1.0):
    """ids [M, top_k] int32 and weights [M, top_k] float64."""
    x = np.asarray(logits, np.float64)
    M, E = x.shape
    gs = E // n_group
    ids = np.empty((M, top_k), np.int32)
    w = np.empty((M, top_k))
    for t in range(M):
        s = _softmax(x[t]) if score == SOFTMAX else _sigmoid(x[t])
        biased = s
        if bias is not None:                 # a logit of -inf masks its expert, whatever its bias
            biased = np.where(x[t] == -np.inf, -np.inf, s + np.asarray(bias, np.float64))
        key = x[t] if bias is None else biased
        worth = np.empty(n_group)
        for g in range(n_group):
            mine = range(g * gs, (g + 1) * gs)
            if group_rule == GROUP_MAX:
                worth[g] = key[_ranked(key, mine)[0]]
            elif gs >= 2:
                a, b = _ranked(biased, mine)[:2]
                worth[g] = _to_38_bits(biased[a] + biased[b])
        kept = range(n_group) if topk_group == n_group else _ranked(worth, range(n_group))[:topk_group]
        pool = [e for g in kept for e in range(g * gs, (g + 1) * gs)]
        chosen = _ranked(key, pool)[:top_k]
        ids[t] = chosen
        if renormalize and score == SOFTMAX:
            v = np.full(top_k, np.nan) if np.isnan(s).any() else _softmax(x[t, chosen])
        else:
            v = s[chosen]
            if renormalize:
                total = v.sum()
                v = np.zeros(top_k) if total == 0 else v / total
        w[t] = v * scale
    return ids, w


def route_backward(d_weights, ids, logits, score=SOFTMAX, renormalize=True, scale=1.0):
    """d_logits [M, E] float64 of the weights of the given choices.  Ids
    outside the experts take no part."""
    x = np.asarray(logits, np.float64)
    dw = np.asarray(d_weights, np.float64)
    M, E = x.shape
    out = np.zeros((M, E))
    for t in range(M):
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        c = np.asarray([ids[t, j] for j in js], np.int64)
        g = dw[t, js]
        if len(js) == 0:
            continue
        if score == SOFTMAX:
            p = _softmax(x[t, c]) if renormalize else _softmax(x[t])[c]
            u = float((g * p).sum())
            if renormalize:
                np.add.at(out[t], c, scale * p * (g - u))
            else:
                np.add.at(out[t], c, scale * p * g)
                out[t] -= scale * u * _softmax(x[t])
        else:
            s = _sigmoid(x[t, c])
            if renormalize:
                total = s.sum()
                if total == 0:
                    continue
                s = s / total                # not g / total: that overflows
                g = g - (g * s).sum()
            np.add.at(out[t], c, scale * g * s * _sigmoid(-x[t, c]))
    return out


def align_ids(ids, E, block_m, expert_first=0):
    """sorted slots, block labels, padded length and counts, as
    oracle.moe.align_block_size with the slots outside the window left out."""
    flat = np.asarray(ids, np.int64).reshape(-1) - expert_first
    S = flat.size
    n = (S + E * (block_m - 1) + block_m - 1) // block_m * block_m
    out = np.full(n, S, np.int32)
    labels = np.full(n // block_m, -1, np.int32)
    counts = np.zeros(E, np.int32)
    at = 0
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        counts[e] = mine.size
        out[at:at + mine.size] = mine
        blocks = (mine.size + block_m - 1) // block_m
        labels[at // block_m:at // block_m + blocks] = e
        at += blocks * block_m
    return out, labels, at, counts


def gemm_int8(a, a_scale, w, w_scale, bias=None, addend=None):
    """(result, sum of the magnitudes of its terms), float64."""
    prod = np.asarray(a, np.float64) @ np.asarray(w, np.float64).T
    prod *= np.asarray(a_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None]
    mag = np.abs(prod)
    if bias is not None:
        prod = prod + np.asarray(bias, np.float64)
        mag = mag + np.abs(np.asarray(bias, np.float64))
    if addend is not None:
        prod = prod + np.asarray(addend, np.float64)
        mag = mag + np.abs(np.asarray(addend, np.float64))
    return prod, mag
