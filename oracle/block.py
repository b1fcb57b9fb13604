"""Reference of the operators of the block around the experts, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The experts' gated feed-forward with its gradients, low-rank adapters of many
requests, and the norms before and after a block with its gate and the
residual.  Each follows its definition expert by expert or token by token.
"""

import numpy as np

SILU, GELU = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2
_C = np.sqrt(2.0 / np.pi)


def _sigmoid(z):
    e = np.exp(-np.abs(z))                       # does not overflow
    return np.where(z < 0, e, 1.0) / (1.0 + e)


def act(g, kind):
    """act(g) and its derivative; their limits at infinite g."""
    g = np.asarray(g, np.float64)
    if kind == SILU:
        z, dz = g, 1.0
    else:
        # (1 + tanh(v)) / 2 = sigmoid(2 v), which does not cancel where tanh is nearly -1
        z = 2.0 * _C * (g + 0.044715 * g ** 3)
        dz = 2.0 * _C * (1.0 + 3.0 * 0.044715 * g * g)
    s = _sigmoid(z)
    with np.errstate(invalid="ignore"):
        a, da = g * s, s + g * s * (1.0 - s) * dz
    return np.where(g == -np.inf, 0.0, a), np.where(np.isinf(g), g > 0, da)


def segments(offsets, rows):
    """[lo, hi) of every expert; offsets outside [0, rows] count as the nearer end."""
    if offsets is None:
        return [(0, rows)]
    out = []
    for e in range(len(offsets) - 1):
        lo = min(max(int(offsets[e]), 0), rows)
        out.append((lo, min(max(int(offsets[e + 1]), lo), rows)))
    return out


def grouped_linear(x, w, segs, out):
    """out[lo:hi] = x[lo:hi] w[e]^T, other rows of `out` as they are."""
    for e, (lo, hi) in enumerate(segs):
        out[lo:hi] = x[lo:hi] @ w[e].T
    return out


def grouped_dgrad(dy, w, segs, out):
    for e, (lo, hi) in enumerate(segs):
        out[lo:hi] = dy[lo:hi] @ w[e]
    return out


def grouped_wgrad(dy, x, segs):
    return np.stack([dy[lo:hi].T @ x[lo:hi] for lo, hi in segs])


def gated_up(x, w, segs, kind, gu, h):
    """gu [rows, 2H] and h [rows, H], written where an expert has rows."""
    H = h.shape[1]
    grouped_linear(x, w, segs, gu)
    for lo, hi in segs:
        h[lo:hi] = act(gu[lo:hi, :H], kind)[0] * gu[lo:hi, H:]
    return gu, h


def gated_down_backward(dy, w, gu, segs, kind, dgu, h):
    H = gu.shape[1] // 2
    for e, (lo, hi) in enumerate(segs):
        a, da = act(gu[lo:hi, :H], kind)
        u = gu[lo:hi, H:]
        dh = dy[lo:hi] @ w[e]
        dgu[lo:hi, :H], dgu[lo:hi, H:], h[lo:hi] = dh * u * da, dh * a, a * u
    return dgu, h


def lora(x, a, b, ids, ranks, scales, addend):
    """addend_t + scales[a] b[a, :, :r] (a[a, :r] x_t), token by token."""
    L, R = a.shape[0], a.shape[1]
    out = np.zeros((x.shape[0], b.shape[1])) if addend is None else np.array(addend, np.float64)
    for t, i in enumerate(np.asarray(ids).reshape(-1)):
        if 0 <= i < L:
            r = R if ranks is None else min(max(int(ranks[i]), 0), R)
            out[t] += (1.0 if scales is None else scales[i]) * (b[i, :, :r] @ (a[i, :r] @ x[t]))
    return out


def norm_residual(y, top_k, residual, w_post, gate, gate_kind, alpha, beta, w_pre, eps, M, N):
    """r, h, rstd_post, rstd_pre (h and the factors None where not taken)."""
    s = np.zeros((M, N)) if y is None else y.reshape(M, top_k, N).sum(1)
    f_post = f_pre = h = None
    p = s
    if w_post is not None:
        f_post = 1.0 / np.sqrt((s * s).mean(1) + eps)
        p = w_post * (s * f_post[:, None])
    if gate_kind != GATE_NONE:
        p = p * (gate[None] if gate_kind == GATE_CHANNEL else gate[:, None])
    r = beta * p + (0.0 if residual is None else alpha * residual)
    if w_pre is not None:
        f_pre = 1.0 / np.sqrt((r * r).mean(1) + eps)
        h = w_pre * (r * f_pre[:, None])
    return r, h, f_post, f_pre


def norm_residual_backward(d_r, d_h, y, top_k, r, w_post, gate, gate_kind, alpha, beta, w_pre,
                           f_post, f_pre, M, N):
    """d_residual, d_y, d_w_post, d_gate, d_w_pre (None for what is not there)."""
    dr = np.zeros((M, N)) if d_r is None else np.array(d_r, np.float64)
    d_y = d_w_post = d_gate = d_w_pre = None
    if w_pre is not None:
        n = r * f_pre[:, None]
        d = d_h * w_pre
        dr = dr + f_pre[:, None] * (d - n * (d * n).mean(1, keepdims=True))
        d_w_pre = (d_h * n).sum(0)
    if y is not None:
        s = y.reshape(M, top_k, N).sum(1)
        m = s if w_post is None else s * f_post[:, None]
        p = m if w_post is None else w_post * m
        dq = beta * dr
        dp = dq
        if gate_kind == GATE_CHANNEL:
            dp, d_gate = dq * gate[None], (dq * p).sum(0)
        elif gate_kind == GATE_TOKEN:
            dp, d_gate = dq * gate[:, None], (dq * p).sum(1)
        d_y = dp
        if w_post is not None:
            d_w_post = (dp * m).sum(0)
            d = dp * w_post
            d_y = f_post[:, None] * (d - m * (d * m).mean(1, keepdims=True))
    return alpha * dr, d_y, d_w_post, d_gate, d_w_pre
