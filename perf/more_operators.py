"""Measured cases of the operators of the block around the experts: the gated
feed-forward of experts in 16 bits with its gradients, low-rank adapters of many
requests beside a shared projection, and the norms before and after the block
fused with its gate and the residual.

Each case names an operator ("op") and its sizes.  `run` computes it in plain
torch operations, or, where `own` is true, with the library's entry points on
the same inputs and the same caller-owned output buffers.
"""

import random

import torch

own = False

F32, BF16, F16 = "f32", "bf16", "f16"
DTYPES = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
CODES = {F32: 0, BF16: 1, F16: 2}                # the library's element type codes
ACTS = {"silu": 0, "gelu": 1}
GATES = {"none": 0, "channel": 1, "token": 2}
EPS = 1e-6
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------
def _ffn(name, rows, K, H, E, dtype, act="silu", train=False, empty=0):
    """Gated feed-forward [rows, K] -> [rows, K] of E experts of width H, of which
    `empty` have no rows; with `train` what the gradient needs is returned too."""
    return {"name": name, "op": "ffn", "rows": rows, "K": K, "H": H, "E": E, "dtype": dtype,
            "act": act, "train": train, "empty": empty}


def _ffn_bwd(name, rows, K, H, E, dtype, act="silu", empty=0):
    return {"name": name, "op": "ffn_backward", "rows": rows, "K": K, "H": H, "E": E,
            "dtype": dtype, "act": act, "empty": empty}


def _lora(name, T, K, N, R, L, dtype, y_dtype, block_m, requests, mixed=False, bare=0.0):
    """T tokens of `requests` requests, each with one of L adapters of rank R (`mixed`:
    up to R) or, a share `bare` of them, with none."""
    return {"name": name, "op": "lora", "T": T, "K": K, "N": N, "R": R, "L": L, "dtype": dtype,
            "y_dtype": y_dtype, "block_m": block_m, "requests": requests, "mixed": mixed,
            "bare": bare}


def _norm(name, op, M, N, top_k, dtype, r_dtype, post=True, gate="none", alpha=1.0, beta=1.0):
    return {"name": name, "op": op, "M": M, "N": N, "top_k": top_k, "dtype": dtype,
            "r_dtype": r_dtype, "post": post, "gate": gate, "alpha": alpha, "beta": beta}


def listed():
    return [
        # one token being decoded, through a shared expert
        _ffn("ffn_one_token", 1, 4096, 14336, 1, BF16),
        # a decode batch of 64 tokens with two experts each
        _ffn("ffn_decode_e8", 128, 4096, 7168, 8, BF16),
        # the experts' forward pass of a training step of 4096 tokens, top 2 of 8
        _ffn("ffn_train_e8", 8192, 4096, 14336, 8, BF16, train=True),
        # a small fine-tuning batch: ragged segments, an expert without rows
        _ffn_bwd("ffn_bwd_ragged", 777, 1024, 1792, 5, F16, "gelu", empty=1),
        # the experts' backward pass of the training step
        _ffn_bwd("ffn_bwd_e8", 8192, 4096, 14336, 8, BF16),
        # one token with an adapter beside a dense projection
        _lora("lora_one_token", 1, 4096, 4096, 16, 8, BF16, BF16, 16, 1),
        # a decode batch of 64 requests, adapters of different ranks, some without
        _lora("lora_decode", 64, 4096, 14336, 64, 32, BF16, BF16, 16, 64, True, 0.1),
        # the prompts of 12 requests at once beside the widest projection
        _lora("lora_prefill", 4096, 4096, 28672, 64, 8, BF16, BF16, 128, 12),
        # one token being decoded, two experts
        _norm("norm_one_token", "norm", 1, 4096, 2, BF16, BF16),
        # a prefill of 4096 tokens, two experts, the block gated per token
        _norm("norm_m4096_k2", "norm", 4096, 4096, 2, BF16, BF16, gate="token", beta=0.5),
        # a small training batch, float32 residual, layer scale, no norm after the block
        _norm("norm_bwd_ragged", "norm_backward", 777, 1792, 1, F16, F32, False, "channel", 1.0, 0.7),
        # a training batch, norms before and after, layer scale
        _norm("norm_bwd_m8192", "norm_backward", 8192, 6144, 1, BF16, BF16, True, "channel"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_backward", "lora", "lora", "norm", "norm_backward"])
    dtype = rng.choice([BF16, BF16, F16])
    if op in ("ffn", "ffn_backward"):
        m = rng.choice([8, 64, 64, 256])
        E = rng.choice([1, 2, 4, 5, 8, 16, 32])
        act = rng.choice(["silu", "gelu"])
        while True:
            rows, K, H = _log(rng, 1, 8192), _mult(rng, 256, 4096, m), _mult(rng, 256, 14336, m)
            if E * K * H <= 8 * 4096 * 14336:
                break
        empty = rng.choice([0, 0, E // 4])
        if op == "ffn":
            c = _ffn("", rows, K, H, E, dtype, act, rng.random() < 0.4, empty)
        else:
            c = _ffn_bwd("", rows, K, H, E, dtype, act, empty)
    elif op == "lora":
        T = _log(rng, 1, 4096)
        m = rng.choice([8, 64, 256])
        block_m = 16 if T < 256 else rng.choice([16, 64, 128])
        c = _lora("", T, _mult(rng, 256, 8192, m), _mult(rng, 256, 28672, m),
                  rng.choice([8, 16, 24, 32, 64, 64, 128]), rng.choice([1, 3, 8, 32, 100]), dtype,
                  rng.choice([dtype, dtype, F32]), block_m, min(T, _log(rng, 1, 64)),
                  rng.random() < 0.5, rng.choice([0.0, 0.0, 0.3]))
        if T * c["N"] > 4096 * 28672 // (2 if c["y_dtype"] == F32 else 1):
            c["N"] = 4096
    else:
        gate = rng.choice(["none", "channel", "token"])
        c = _norm("", op, _log(rng, 1, 8192), _mult(rng, 128, 6144, rng.choice([8, 64, 256])),
                  rng.choice([1, 1, 2, 4]) if op == "norm" else rng.choice([1, 1, 2]), dtype,
                  rng.choice([dtype, F32]), rng.random() < 0.6, gate,
                  rng.choice([1.0, 1.0, 0.8]), rng.choice([1.0, 0.5]))
        if c["op"] == "norm" and c["top_k"] == 4:
            c["M"] = min(c["M"], 4096)
        if c["op"] == "norm_backward" and c["top_k"] == 2:
            c["M"] = min(c["M"], 4096)
        if c["r_dtype"] == F32:
            c["M"] = min(c["M"], 4096)
    del c["name"]
    return c


# ---- plans made on the host from the seed --------------------------------------------
def _splits(c, seed):
    """Rows of every expert: uneven, the empty ones anywhere."""
    rng = random.Random(seed * 7919 + 11)
    E, rows = c["E"], c["rows"]
    gone = set(rng.sample(range(E), c["empty"]))
    share = [0.0 if e in gone else 0.5 + rng.random() for e in range(E)]
    total, cut, out, acc = sum(share), 0, [], 0.0
    for e in range(E):
        acc += share[e]
        nxt = int(rows * acc / total + 0.5)
        out.append(nxt - cut)
        cut = nxt
    last = max(e for e in range(E) if e not in gone)
    out[last] += rows - cut
    return out


def _requests(c, seed):
    """(adapter or -1, tokens) of every request, and the adapters' ranks."""
    rng = random.Random(seed * 104729 + 5)
    n, T = c["requests"], c["T"]
    cuts = [0] + sorted(rng.sample(range(1, T), n - 1)) + [T] if n > 1 else [0, T]
    reqs = []
    for i in range(n):
        bare = rng.random() < c["bare"]
        reqs.append((-1 if bare else rng.randrange(c["L"]), cuts[i + 1] - cuts[i]))
    ranks = [rng.randint(1, c["R"]) if c["mixed"] else c["R"] for _ in range(c["L"])]
    return reqs, ranks


def _padded(T, L, block_m):
    n = T + L * (block_m - 1)
    return (n + block_m - 1) // block_m * block_m


def work(c):
    """Inputs read once, outputs written once (weights of the experts and adapters
    that have tokens); operations: a multiply and an add each."""
    if c["op"] in ("ffn", "ffn_backward"):
        rows, K, H, E = c["rows"], c["K"], c["H"], c["E"]
        used = min(rows, E - c["empty"])
        mac = 3 * rows * K * H
        weights = 3 * K * H * 2
        if c["op"] == "ffn":
            kept = 6 * rows * H * c["train"]                  # gu and h
            return {"bytes": used * weights + 4 * rows * K + kept, "flops": 2 * mac}
        return {"bytes": used * weights + E * weights + 2 * rows * (3 * K + 2 * H),
                "flops": 4 * mac}
    if c["op"] == "lora":
        T, K, N, R = c["T"], c["K"], c["N"], c["R"]
        y = 4 if c["y_dtype"] == F32 else 2
        used = min(c["L"], c["requests"])
        r = R // 2 if c["mixed"] else R
        return {"bytes": T * K * 2 + used * r * (K + N) * 2 + 2 * T * N * y,
                "flops": 2 * T * r * (K + N)}
    M, N, k = c["M"], c["N"], c["top_k"]
    r = 4 if c["r_dtype"] == F32 else 2
    if c["op"] == "norm":
        return {"bytes": M * N * (2 * k + 2 + 2 * r), "flops": M * N * (k + 10)}
    return {"bytes": M * N * (2 * k + 4 + 3 * r), "flops": M * N * (k + 25)}


# ---- inputs ---------------------------------------------------------------------
def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def prepare(c, seed):
    seed = int(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c)
    t = DTYPES[c["dtype"]]

    def randn(*shape, std=1.0, dtype=t):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(std)

    if c["op"] in ("ffn", "ffn_backward"):
        rows, K, H, E = c["rows"], c["K"], c["H"], c["E"]
        s["splits"] = _splits(c, seed)
        at = [0]
        for n in s["splits"]:
            at.append(at[-1] + n)
        s["off"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        s["x"] = randn(rows, K)                              # rows behind a norm
        s["w_up"] = randn(E, 2 * H, K, std=K ** -0.5)
        s["w_down"] = randn(E, K, H, std=H ** -0.5)
        s["h"] = _empty(rows, H, dtype=t)
        if c["op"] == "ffn":
            s["gu"] = _empty(rows, 2 * H, dtype=t) if c["train"] else None
            s["y"] = _empty(rows, K, dtype=t)
        else:
            s["dy"] = randn(rows, K, std=0.02)
            s["gu"] = randn(rows, 2 * H)                     # as the forward pass left them
            s["dgu"] = _empty(rows, 2 * H, dtype=t)
            s["dx"] = _empty(rows, K, dtype=t)
            s["dw_up"] = _empty(E, 2 * H, K, dtype=t)
            s["dw_down"] = _empty(E, K, H, dtype=t)
    elif c["op"] == "lora":
        T, K, N, R, L, b = c["T"], c["K"], c["N"], c["R"], c["L"], c["block_m"]
        reqs, ranks = _requests(c, seed)
        ids = []
        for a, n in reqs:
            ids += [a] * n
        s["reqs"], s["rank_list"] = reqs, ranks
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
        s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device=DEV)
        s["scales"] = torch.rand(L, generator=g, device=DEV) + 0.5
        s["x"] = randn(T, K)
        s["a"] = randn(L, R, K, std=K ** -0.5)
        s["b"] = randn(L, N, R, std=R ** -0.5)
        s["y0"] = randn(T, N, dtype=DTYPES[c["y_dtype"]])    # the shared projection's output
        s["y"] = _empty(T, N, dtype=DTYPES[c["y_dtype"]])
        # the tokens grouped by adapter, once for all projections of a step
        order, labels = [], []
        for a in range(L):
            mine = [i for i, v in enumerate(ids) if v == a]
            blocks = (len(mine) + b - 1) // b
            order += mine + [T] * (blocks * b - len(mine))
            labels += [a] * blocks
        n = _padded(T, L, b)
        s["post"] = torch.tensor([len(order)], dtype=torch.int32, device=DEV)
        s["sorted"] = torch.tensor(order + [T] * (n - len(order)), dtype=torch.int32, device=DEV)
        s["labels"] = torch.tensor(labels + [-1] * (n // b - len(labels)), dtype=torch.int32,
                                   device=DEV)
        s["ws"] = _empty(64 << 20, dtype=torch.uint8)        # scratch that the caller keeps
    else:
        M, N, k, rt = c["M"], c["N"], c["top_k"], DTYPES[c["r_dtype"]]
        s["y"] = randn(M * k, N)                             # the experts' results, slot by slot
        s["w_pre"] = 1.0 + 0.2 * torch.randn(N, generator=g, device=DEV)
        s["w_post"] = 0.3 + 0.1 * torch.randn(N, generator=g, device=DEV) if c["post"] else None
        shape = {"none": 0, "channel": N, "token": M}[c["gate"]]
        s["gate_v"] = torch.rand(shape, generator=g, device=DEV) + 0.1 if shape else None
        if c["op"] == "norm":
            s["x"] = randn(M, N, std=2.0, dtype=rt)
            s["r"], s["h"] = _empty(M, N, dtype=rt), _empty(M, N, dtype=t)
            s["rstd_post"] = _empty(M) if c["post"] else None
            s["rstd_pre"] = _empty(M)
        else:
            # what the forward pass left: the new residual and both norms' factors
            r = randn(M, N, std=2.0, dtype=torch.float32)
            s["rstd_pre"] = torch.rsqrt((r * r).mean(1) + EPS)
            s["r"] = r.to(rt)
            s["rstd_post"] = None
            if c["post"]:
                y = s["y"].view(M, k, N).float().sum(1)
                s["rstd_post"] = torch.rsqrt((y * y).mean(1) + EPS)
            s["dr"] = randn(M, N, dtype=rt)
            s["dh"] = randn(M, N)
            s["dx"], s["dy"] = _empty(M, N, dtype=rt), _empty(M, N, dtype=t)
            s["dw_post"] = _empty(N) if c["post"] else None
            s["dw_pre"] = _empty(N)
            s["d_gate"] = _empty(shape) if shape else None
            s["ws"] = _empty(64 << 20, dtype=torch.uint8)    # scratch that the caller keeps
    return s


# ---- plain forms ------------------------------------------------------------------
GELU_C = 0.7978845608028654


def _act(x, act):
    """act(x) and its derivative."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return x * p, p * (1.0 + x * (1.0 - p))
    z = 2.0 * GELU_C * (x + 0.044715 * x * x * x)
    p = 1.0 / (1.0 + torch.exp(-z))
    return x * p, p + x * p * (1.0 - p) * (2.0 * GELU_C * (1.0 + 3.0 * 0.044715 * x * x))


def _segments(s):
    lo = 0
    for e, n in enumerate(s["splits"]):
        yield e, slice(lo, lo + n), n
        lo += n


def _plain_ffn(s):
    H, t = s["H"], DTYPES[s["dtype"]]
    y = torch.empty_like(s["y"])
    gu = torch.empty_like(s["gu"]) if s["train"] else None
    h = torch.empty_like(s["h"]) if s["train"] else None
    for e, seg, n in _segments(s):
        if not n:
            continue
        p = s["x"][seg].float() @ s["w_up"][e].float().t()
        v = _act(p[:, :H], s["act"])[0] * p[:, H:]
        y[seg] = (v @ s["w_down"][e].float().t()).to(t)
        if s["train"]:
            gu[seg], h[seg] = p.to(t), v.to(t)
    return (y, gu, h) if s["train"] else y


def _plain_ffn_backward(s):
    H, t = s["H"], DTYPES[s["dtype"]]
    dx, dw_up, dw_down = (torch.empty_like(s[k]) for k in ("dx", "dw_up", "dw_down"))
    for e, seg, n in _segments(s):
        x, dy, gu = s["x"][seg].float(), s["dy"][seg].float(), s["gu"][seg].float()
        a, da = _act(gu[:, :H], s["act"])
        dh = dy @ s["w_down"][e].float()
        d = torch.cat([dh * gu[:, H:] * da, dh * a], dim=1)
        dx[seg] = (d @ s["w_up"][e].float()).to(t)
        dw_up[e] = (d.t() @ x).to(t)
        dw_down[e] = (dy.t() @ (a * gu[:, H:])).to(t)
    return dx, dw_up, dw_down


def _plain_lora(s):
    out = s["y0"].clone()
    lo = 0
    for a, n in s["reqs"]:
        if a >= 0:
            r = s["rank_list"][a]
            v = s["x"][lo:lo + n].float() @ s["a"][a, :r].float().t()
            d = (v @ s["b"][a, :, :r].float().t()) * s["scales"][a]
            out[lo:lo + n] = (s["y0"][lo:lo + n].float() + d).to(out.dtype)
        lo += n
    return out


def _gate_of(s):
    if s["gate_v"] is None:
        return 1.0
    return s["gate_v"][None] if s["gate"] == "channel" else s["gate_v"][:, None]


def _plain_norm(s):
    M, N, k = s["M"], s["N"], s["top_k"]
    p = s["y"].view(M, k, N).float().sum(1)
    rstd_post = None
    if s["post"]:
        rstd_post = torch.rsqrt((p * p).mean(1) + EPS)
        p = p * rstd_post[:, None] * s["w_post"]
    r = s["alpha"] * s["x"].float() + s["beta"] * (_gate_of(s) * p)
    rstd = torch.rsqrt((r * r).mean(1) + EPS)
    h = r * rstd[:, None] * s["w_pre"]
    out = (r.to(s["r"].dtype), h.to(s["h"].dtype), rstd)
    return out + (rstd_post,) if s["post"] else out


def _plain_norm_backward(s):
    M, N, k = s["M"], s["N"], s["top_k"]
    n = s["r"].float() * s["rstd_pre"][:, None]
    dh = s["dh"].float()
    d = dh * s["w_pre"]
    dr = s["dr"].float() + s["rstd_pre"][:, None] * (d - n * (d * n).mean(1, keepdim=True))
    out = [(s["alpha"] * dr).to(s["dx"].dtype), None, (dh * n).sum(0)]
    y = s["y"].view(M, k, N).float().sum(1)
    dq = s["beta"] * dr
    dp = _gate_of(s) * dq
    p = y
    if s["post"]:
        yn = y * s["rstd_post"][:, None]
        p = yn * s["w_post"]
        out.append((dp * yn).sum(0))
        d = dp * s["w_post"]
        dp = s["rstd_post"][:, None] * (d - yn * (d * yn).mean(1, keepdim=True))
    if s["gate"] != "none":
        out.append((dq * p).sum(0 if s["gate"] == "channel" else 1))
    out[1] = dp.to(s["dy"].dtype)
    return tuple(out)


# ---- one pass -----------------------------------------------------------------------
def _own_ffn(s):
    import quantized_moe_grouped_top_amd as qm
    t, rows, K, H, E = CODES[s["dtype"]], s["rows"], s["K"], s["H"], s["E"]
    qm.moe_gated_up(s["x"], K, s["w_up"], t, s["off"], rows, K, H, E, ACTS[s["act"]], s["gu"], s["h"])
    qm.moe_grouped_linear(s["h"], H, s["w_down"], t, s["off"], rows, H, K, E, s["y"], K)
    return (s["y"], s["gu"], s["h"]) if s["train"] else s["y"]


def _own_ffn_backward(s):
    import quantized_moe_grouped_top_amd as qm
    t, rows, K, H, E = CODES[s["dtype"]], s["rows"], s["K"], s["H"], s["E"]
    off = s["off"]
    qm.moe_gated_down_backward(s["dy"], K, s["w_down"], s["gu"], t, off, rows, K, H, E,
                               ACTS[s["act"]], s["dgu"], s["h"])
    qm.moe_grouped_linear_dgrad(s["dgu"], 2 * H, s["w_up"], t, off, rows, K, 2 * H, E, s["dx"], K)
    qm.moe_grouped_linear_wgrad(s["dgu"], 2 * H, s["x"], K, t, off, rows, K, 2 * H, E, t, s["dw_up"])
    qm.moe_grouped_linear_wgrad(s["dy"], K, s["h"], H, t, off, rows, H, K, E, t, s["dw_down"])
    return s["dx"], s["dw_up"], s["dw_down"]


def _own_lora(s):
    import quantized_moe_grouped_top_amd as qm
    qm.moe_lora_add(s["x"], s["K"], s["a"], s["b"], s["ranks"], s["scales"], CODES[s["dtype"]],
                    s["ids"], s["sorted"], s["labels"], s["post"], s["T"], s["K"], s["N"], s["R"],
                    s["L"], s["block_m"], s["y0"], CODES[s["y_dtype"]], s["y"], s["N"], s["ws"])
    return s["y"]


def _own_norm(s):
    import quantized_moe_grouped_top_amd as qm
    qm.moe_norm_residual(s["y"], CODES[s["dtype"]], s["top_k"], s["x"], CODES[s["r_dtype"]],
                         s["w_post"], s["gate_v"], GATES[s["gate"]], s["alpha"], s["beta"],
                         s["w_pre"], EPS, s["M"], s["N"], s["r"], s["h"], s["rstd_post"],
                         s["rstd_pre"])
    out = (s["r"], s["h"], s["rstd_pre"])
    return out + (s["rstd_post"],) if s["post"] else out


def _own_norm_backward(s):
    import quantized_moe_grouped_top_amd as qm
    qm.moe_norm_residual_backward(s["dr"], s["dh"], s["y"], CODES[s["dtype"]], s["top_k"], s["r"],
                                  CODES[s["r_dtype"]], s["w_post"], s["gate_v"], GATES[s["gate"]],
                                  s["alpha"], s["beta"], s["w_pre"], s["rstd_post"], s["rstd_pre"],
                                  s["M"], s["N"], s["dx"], s["dy"], s["dw_post"], s["d_gate"],
                                  s["dw_pre"], s["ws"])
    out = [s["dx"], s["dy"], s["dw_pre"]]
    if s["post"]:
        out.append(s["dw_post"])
    if s["gate"] != "none":
        out.append(s["d_gate"])
    return tuple(out)


PLAIN = {"ffn": _plain_ffn, "ffn_backward": _plain_ffn_backward, "lora": _plain_lora,
         "norm": _plain_norm, "norm_backward": _plain_norm_backward}
OWN = {"ffn": _own_ffn, "ffn_backward": _own_ffn_backward, "lora": _own_lora, "norm": _own_norm,
       "norm_backward": _own_norm_backward}


def run(s):
    if own:
        return OWN[s["op"]](s)
    return PLAIN[s["op"]](s)


# ---- definitions in 64 bits ------------------------------------------------------------
def _exact_gated(a, b, act):
    """act(a) * b with the textbook forms: sigmoid, tanh."""
    if act == "silu":
        return a * torch.sigmoid(a) * b
    return 0.5 * a * (1.0 + torch.tanh(GELU_C * (a + 0.044715 * a ** 3))) * b


def _exact_ffn(c, s):
    H = c["H"]
    y = torch.empty(c["rows"], c["K"], dtype=torch.float64, device=DEV)
    gu = torch.empty(c["rows"], 2 * H, dtype=torch.float64, device=DEV) if c["train"] else None
    h = torch.empty(c["rows"], H, dtype=torch.float64, device=DEV) if c["train"] else None
    off = s["off"].tolist()
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        x = s["x"][lo:hi].double()
        a = torch.matmul(x, s["w_up"][e, :H].double().t())
        b = torch.matmul(x, s["w_up"][e, H:].double().t())
        v = _exact_gated(a, b, c["act"])
        y[lo:hi] = torch.matmul(v, s["w_down"][e].double().t())
        if c["train"]:
            gu[lo:hi, :H], gu[lo:hi, H:], h[lo:hi] = a, b, v
    return (y, gu, h) if c["train"] else y


def _exact_ffn_backward(c, s):
    """By the chain rule through h, the activation's derivative by differentiation."""
    H, off = c["H"], s["off"].tolist()
    dx = torch.empty(c["rows"], c["K"], dtype=torch.float64, device=DEV)
    dw_up = torch.zeros(c["E"], 2 * H, c["K"], dtype=torch.float64, device=DEV)
    dw_down = torch.zeros(c["E"], c["K"], H, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        dy = s["dy"][lo:hi].double()
        with torch.enable_grad():
            gu = s["gu"][lo:hi].double().requires_grad_(True)
            h = _exact_gated(gu[:, :H], gu[:, H:], c["act"])
            dgu, = torch.autograd.grad(h, gu, torch.matmul(dy, s["w_down"][e].double()))
        dx[lo:hi] = torch.matmul(dgu, s["w_up"][e].double())
        dw_up[e] = torch.matmul(dgu.t(), s["x"][lo:hi].double())
        dw_down[e] = torch.matmul(dy.t(), h.detach())
    return dx, dw_up, dw_down


def _exact_lora(c, s):
    y = s["y0"].double()
    ids, ranks = s["ids"].tolist(), s["ranks"].tolist()
    for a in sorted(set(ids) - {-1}):
        at = torch.tensor([i for i, v in enumerate(ids) if v == a], device=DEV)
        product = torch.matmul(s["b"][a, :, :ranks[a]].double(),
                               torch.matmul(s["a"][a, :ranks[a]].double(), s["x"][at].double().t()))
        y[at] += s["scales"][a].double() * product.t()
    return y


def _exact_factors(c, s):
    gate = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    if c["gate"] == "channel":
        gate = s["gate_v"].double().reshape(1, -1)
    if c["gate"] == "token":
        gate = s["gate_v"].double().reshape(-1, 1)
    y = s["y"].double().reshape(c["M"], c["top_k"], c["N"])
    total = y[:, 0]
    for j in range(1, c["top_k"]):
        total = total + y[:, j]
    return gate, total


def _exact_norm(c, s):
    gate, p = _exact_factors(c, s)
    N = c["N"]
    f_post = None
    if c["post"]:
        f_post = 1.0 / (torch.linalg.vector_norm(p, dim=1) ** 2 / N + EPS).sqrt()
        p = s["w_post"].double() * (p * f_post.unsqueeze(1))
    r = s["x"].double() * c["alpha"] + gate * p * c["beta"]
    f = 1.0 / (torch.linalg.vector_norm(r, dim=1) ** 2 / N + EPS).sqrt()
    out = (r, s["w_pre"].double() * (r * f.unsqueeze(1)), f)
    return out + (f_post,) if c["post"] else out


def _exact_norm_backward(c, s):
    """With the given factors held as 1 / rms: d rstd / d r = -rstd^3 r / N."""
    gate, total = _exact_factors(c, s)
    N = c["N"]
    r, f = s["r"].double(), s["rstd_pre"].double().unsqueeze(1)
    dh, w = s["dh"].double(), s["w_pre"].double()
    dot = torch.einsum("mn,mn->m", dh * w, r).unsqueeze(1)
    dr = s["dr"].double() + f * w * dh - f ** 3 * r * dot / N
    dw_pre = torch.einsum("mn,mn->n", dh, r * f)
    dq = dr * c["beta"]
    dp, p, tail = dq * gate, total, []
    if c["post"]:
        fp, wp = s["rstd_post"].double().unsqueeze(1), s["w_post"].double()
        p = wp * total * fp
        tail.append(torch.einsum("mn,mn->n", dp, total * fp))
        dot = torch.einsum("mn,mn->m", dp * wp, total).unsqueeze(1)
        dp = fp * wp * dp - fp ** 3 * total * dot / N
    if c["gate"] == "channel":
        tail.append(torch.einsum("mn,mn->n", dq, p))
    if c["gate"] == "token":
        tail.append(torch.einsum("mn,mn->m", dq, p))
    return (dr * c["alpha"], dp, dw_pre) + tuple(tail)


def exact(c, seed):
    s = prepare(c, seed)
    return {"ffn": _exact_ffn, "ffn_backward": _exact_ffn_backward, "lora": _exact_lora,
            "norm": _exact_norm, "norm_backward": _exact_norm_backward}[c["op"]](c, s)
