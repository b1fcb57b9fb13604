"""Measured cases of the MoE layer's router, its gradient, the block alignment
of its choices and the dense int8 product of the layers beside the experts.

Each case names an operator ("op") and its sizes.  `run` computes it in plain
torch operations, or, where `own` is true, with the library's entry point on
the same inputs and the same caller-owned output buffers.
"""

import torch

own = False

F32, BF16, F16 = "f32", "bf16", "f16"
DTYPES = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
CODES = {F32: 0, BF16: 1, F16: 2}                # the library's element type codes
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_RULES = {"max": 0, "top2": 1}
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------
def _route(name, M, E, top_k, dtype, score, bias=False, groups=1, keep=1, rule="max",
           renorm=True, scale=1.0, pad=0, dead=0):
    return {"name": name, "op": "route", "M": M, "E": E, "top_k": top_k, "dtype": dtype,
            "score": score, "bias": bias, "groups": groups, "keep": keep, "rule": rule,
            "renorm": renorm, "scale": scale, "pad": pad, "dead": dead}


def _route_bwd(name, M, E, top_k, dtype, score, renorm=True, scale=1.0, pad=0):
    return {"name": name, "op": "route_backward", "M": M, "E": E, "top_k": top_k, "dtype": dtype,
            "score": score, "renorm": renorm, "scale": scale, "pad": pad}


def _align(name, M, E, top_k, block_m, first=0, total=None):
    return {"name": name, "op": "align", "M": M, "E": E, "top_k": top_k, "block_m": block_m,
            "first": first, "total": total or E}


def _int8(name, M, K, N, out, bias=False, addend=False, pad=0):
    return {"name": name, "op": "int8", "M": M, "K": K, "N": N, "out": out, "bias": bias,
            "addend": addend, "pad": pad}


def listed():
    return [
        # one token being decoded: sigmoid scores, balance bias, 4 of 8 groups
        _route("route_one_token", 1, 128, 8, F32, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # a prefill of 4096 tokens, bf16 logits as the router's product leaves them
        _route("route_m4096_softmax_bf16", 4096, 128, 8, BF16, "softmax"),
        # a training batch with balance bias and groups
        _route("route_m16384_groups", 16384, 256, 8, F32, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # gradients of a training batch: only the chosen experts / every expert
        _route_bwd("route_bwd_m4096_sigmoid", 4096, 128, 8, BF16, "sigmoid", True, 2.5),
        _route_bwd("route_bwd_m16384_dense", 16384, 256, 8, F32, "softmax", False),
        # the decode shape of the benchmark, and the most slots one call takes
        _align("align_m64", 64, 8, 2, 16),
        _align("align_m8192_e128", 8192, 128, 8, 128),
        # one token through a dense projection
        _int8("int8_m1_k4096_n4096", 1, 4096, 4096, BF16),
        # a decode batch through the shared expert, added to the routed experts' sum
        _int8("int8_m64_k4096_n14336", 64, 4096, 14336, BF16, addend=True),
        # odd sizes, rows padded apart, float32 results with a bias
        _int8("int8_ragged_m777", 777, 1531, 4099, F32, bias=True, pad=5),
        # the up and the down projection of a prefill
        _int8("int8_m4096_k14336_n4096", 4096, 14336, 4096, BF16),
        _int8("int8_m4096_k4096_n28672", 4096, 4096, 28672, BF16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "align", "int8", "int8", "int8"])
    if op == "int8":
        while True:
            M, K, N = _log(rng, 1, 4096), _log(rng, 64, 14336), _log(rng, 64, 28672)
            if M * K * N <= 4096 * 4096 * 28672:
                break
        align = rng.choice([1, 16, 16, 64, 128])       # K and N of real layers are mostly round
        K, N = max(align, K // align * align), max(8, N // align * align)
        c = _int8("", M, K, N, rng.choice([BF16, BF16, F16, F32]), rng.random() < 0.5,
                  rng.random() < 0.4, rng.choice([0, 0, (-K) % 16, 16]))
    else:
        E = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256, 384, 512])
        top_k = rng.randint(1, 8)
        M = _log(rng, 1, 16384)
        dtype = rng.choice([F32, BF16, F16])
        score = rng.choice(["softmax", "sigmoid"])
        scale = rng.choice([1.0, 2.5])
        if op == "route":
            groups, keep, rule = 1, 1, "max"
            if rng.random() < 0.5:
                groups = rng.choice([g for g in (2, 4, 8, 16) if E % g == 0 and E // g >= 2])
                keep = rng.randint(1, groups)
                rule = rng.choice(["max", "top2"])
            top_k = min(top_k, E // groups * keep)
            c = _route("", M, E, top_k, dtype, score, rng.random() < 0.6, groups, keep, rule,
                       rng.random() < 0.7, scale, rng.choice([0, 0, 3, 8]),
                       rng.choice([0, 0, 0, E // 4]))
        elif op == "route_backward":
            renorm = rng.random() < 0.7
            if renorm:                   # one renormalised weight is a constant: no gradient
                top_k = max(2, top_k)
            c = _route_bwd("", M, E, top_k, dtype, score, renorm, scale, rng.choice([0, 0, 3, 8]))
        else:
            E = min(E, 128)
            total = E * rng.choice([1, 1, 1, 2, 4])    # the other experts live elsewhere
            M = min(M, 65536 // top_k)
            c = _align("", M, E, top_k, rng.choice([16, 32, 64, 128, 256]),
                       E * rng.randrange(total // E), total)
    del c["name"]
    return c


def work(c):
    """Inputs read once, outputs written once; operations counted as multiply
    and add (int8), or per score and gradient value (routing)."""
    if c["op"] == "int8":
        M, K, N = c["M"], c["K"], c["N"]
        o = 4 if c["out"] == F32 else 2
        b = M * K + N * K + 4 * (M + N) + 4 * N * c["bias"] + M * N * o * (1 + c["addend"])
        return {"bytes": b, "flops": 2 * M * K * N}
    M, E, k = c["M"], c["E"], c["top_k"]
    if c["op"] == "align":
        S = M * k
        n = _padded(c)
        return {"bytes": 4 * S + 4 * n + 4 * (n // c["block_m"]) + 4 + 4 * E, "flops": S}
    x = 4 if c["dtype"] == F32 else 2
    if c["op"] == "route":
        return {"bytes": M * E * x + 4 * E * c["bias"] + 8 * M * k, "flops": 10 * M * E}
    dense = c["score"] == "softmax" and not c["renorm"]
    return {"bytes": M * E * x * (1 + dense) + M * k * (8 + (0 if dense else x)),
            "flops": 10 * M * (E if dense else k)}


# ---- inputs ---------------------------------------------------------------------
def _logits(c, g):
    ld = c["E"] + c["pad"]
    x = torch.randn(c["M"], ld, generator=g, device=DEV) + \
        0.5 * torch.randn(ld, generator=g, device=DEV)
    return x.to(DTYPES[c["dtype"]])[:, :c["E"]]


def _padded(c):
    n = c["M"] * c["top_k"] + c["E"] * (c["block_m"] - 1)
    return (n + c["block_m"] - 1) // c["block_m"] * c["block_m"]


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(c)
    M = c["M"]
    if c["op"] == "route":
        s["x"] = _logits(c, g)
        s["b"] = None
        if c["bias"]:                    # the bias that keeps the loads even
            s["b"] = 0.1 * torch.randn(c["E"], generator=g, device=DEV)
        if c["dead"]:                    # experts taken out of service
            gone = torch.randperm(c["E"], generator=g, device=DEV)[:c["dead"]]
            if c["bias"]:
                s["b"][gone] = float("-inf")
            else:
                s["x"][:, gone] = float("-inf")
        s["ids"] = _empty(M, c["top_k"], dtype=torch.int32)
        s["w"] = _empty(M, c["top_k"])
    elif c["op"] == "route_backward":
        s["x"] = _logits(c, g)
        noise = torch.rand(M, c["E"], generator=g, device=DEV)
        s["ids"] = (s["x"].float() + noise).topk(c["top_k"], dim=1).indices.int().contiguous()
        s["dw"] = torch.randn(M, c["top_k"], generator=g, device=DEV)
        s["dx"] = _empty(M, c["E"], dtype=DTYPES[c["dtype"]])
    elif c["op"] == "align":
        x = torch.randn(M, c["total"], generator=g, device=DEV) + \
            0.5 * torch.randn(c["total"], generator=g, device=DEV)
        s["ids"] = x.topk(c["top_k"], dim=1).indices.int().contiguous()
        n = _padded(c)
        s["sorted"] = _empty(n, dtype=torch.int32)
        s["labels"] = _empty(n // c["block_m"], dtype=torch.int32)
        s["post"] = _empty(1, dtype=torch.int32)
        s["counts"] = _empty(c["E"], dtype=torch.int32)
        # scratch that the caller keeps: one count for each 1024 slots and expert at most
        s["ws"] = _empty((M * c["top_k"] + 1023) // 1024 * c["E"], dtype=torch.int32)
    else:
        K, N, ld = c["K"], c["N"], c["K"] + c["pad"]

        def codes(rows):
            v = torch.randn(rows, ld, generator=g, device=DEV).mul_(36.0).round_().clamp_(-127, 127)
            return v.to(torch.int8)[:, :K]

        s["a"], s["wq"] = codes(M), codes(N)
        s["sa"] = torch.rand(M, generator=g, device=DEV) * 0.02 + 0.02
        s["sw"] = (torch.rand(N, generator=g, device=DEV) + 1.0) * (0.02 / K ** 0.5)
        s["bias_v"] = torch.randn(N, generator=g, device=DEV) if c["bias"] else None
        o = DTYPES[c["out"]]
        s["add"] = torch.randn(M, N, generator=g, device=DEV).to(o) if c["addend"] else None
        s["y"] = _empty(M, N, dtype=o)
        s["ws"] = _empty(64 << 20, dtype=torch.uint8)      # scratch that the caller keeps
    return s


# ---- plain forms ------------------------------------------------------------------
def _scores(x, score):
    """Scores in float64: which of two close keys is larger is decided here."""
    x = x.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(dim=1, keepdim=True)
    e = torch.where(torch.isinf(m), 0.0, torch.exp(x - m))
    z = e.sum(dim=1, keepdim=True)
    return e / torch.where(z > 0, z, 1.0)


def _plain_route(s):
    M, E, k, n = s["M"], s["E"], s["top_k"], s["groups"]
    p = _scores(s["x"], s["score"])
    biased = p if s["b"] is None else p + s["b"].double()
    key = s["x"].double() if s["b"] is None else biased
    order = key.sort(dim=1, descending=True, stable=True).indices
    if n > 1:
        if s["rule"] == "top2":
            best = biased.view(M, n, E // n).sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        else:
            best = key.view(M, n, E // n).amax(dim=2)
        rank = best.sort(dim=1, descending=True, stable=True).indices
        out = torch.ones(M, n, dtype=torch.int32, device=DEV)
        out.scatter_(1, rank[:, :s["keep"]], 0)
        gone = out.repeat_interleave(E // n, dim=1).gather(1, order)
        order = order.gather(1, gone.sort(dim=1, stable=True).indices)
    ids = order[:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        z = w.sum(dim=1, keepdim=True)
        w = w / torch.where(z > 0, z, 1.0)
    return ids.int(), (w * s["scale"]).float()


def _plain_route_backward(s):
    ids, dw = s["ids"].long(), s["dw"]
    x = s["x"].float()
    if s["score"] == "softmax" and not s["renorm"]:
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        u = (dw * p.gather(1, ids)).sum(dim=1, keepdim=True)
        up = torch.zeros_like(x).scatter_(1, ids, dw)
        return (p * (up - u) * s["scale"]).to(s["dx"].dtype)
    v = x.gather(1, ids)
    if s["score"] == "softmax":
        e = torch.exp(v - v.amax(dim=1, keepdim=True))
        q = e / e.sum(dim=1, keepdim=True)
        d = q * (dw - (dw * q).sum(dim=1, keepdim=True))
    else:
        p = 1.0 / (1.0 + torch.exp(-v))
        d = p * (1.0 / (1.0 + torch.exp(v)))
        if s["renorm"]:
            z = p.sum(dim=1, keepdim=True)
            d = d * (dw - (dw * p).sum(dim=1, keepdim=True) / z) / z
        else:
            d = d * dw
    return torch.zeros_like(x).scatter_(1, ids, d * s["scale"]).to(s["dx"].dtype)


def _plain_align(s):
    E, b, S = s["E"], s["block_m"], s["M"] * s["top_k"]
    e = s["ids"].view(-1).long() - s["first"]
    e = torch.where((e >= 0) & (e < E), e, E)
    counts = (e[:, None] == torch.arange(E, device=DEV)).sum(dim=0)
    size = (counts + b - 1) // b * b
    end = size.cumsum(0)
    order = e.sort(stable=True).indices
    es = e[order]
    starts = torch.cat([end - size, end[-1:]])
    firsts = torch.cat([counts.cumsum(0) - counts, counts.sum()[None]])
    place = starts[es] + torch.arange(S, device=DEV) - firsts[es]
    n = s["sorted"].numel()
    out = torch.full((n + S,), S, dtype=torch.int32, device=DEV)
    place = torch.where(es < E, place, n + torch.arange(S, device=DEV))
    out[place] = order.int()
    out[n:] = S
    at = torch.arange(n // b, device=DEV) * b
    label = (at[:, None] >= end).sum(dim=1)
    label = torch.where(label < E, label, -1)
    return out[:n], label.int(), end[-1:].int(), counts.int()


def _plain_int8(s):
    y = s["a"].float() @ s["wq"].float().t()
    y = y * s["sa"][:, None] * s["sw"]
    if s["bias_v"] is not None:
        y = y + s["bias_v"]
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(s["y"].dtype)


# ---- one pass -----------------------------------------------------------------------
def _own_route(s):
    import quantized_moe_grouped_top_amd as qm
    qm.moe_route_topk(s["x"], CODES[s["dtype"]], s["E"] + s["pad"], s["b"], s["M"], s["E"],
                      s["top_k"], SCORES[s["score"]], s["groups"], s["keep"],
                      GROUP_RULES[s["rule"]], s["renorm"], s["scale"], s["ids"], s["w"])
    return s["ids"], s["w"]


def _own_route_backward(s):
    import quantized_moe_grouped_top_amd as qm
    qm.moe_route_topk_backward(s["dw"], s["ids"], s["x"], CODES[s["dtype"]], s["E"] + s["pad"],
                               s["M"], s["E"], s["top_k"], SCORES[s["score"]], s["renorm"],
                               s["scale"], s["dx"], s["E"])
    return s["dx"]


def _own_align(s):
    import quantized_moe_grouped_top_amd as qm
    qm.moe_align_topk_ids(s["ids"], s["M"], s["E"], s["top_k"], s["block_m"], s["first"],
                          s["sorted"], s["labels"], s["post"], s["counts"], s["ws"])
    return s["sorted"], s["labels"], s["post"], s["counts"]


def _own_int8(s):
    import quantized_moe_grouped_top_amd as qm
    ld = s["K"] + s["pad"]
    qm.moe_gemm_int8w8a8(s["a"], ld, s["sa"], s["wq"], ld, s["sw"], s["bias_v"], s["add"], s["M"],
                         s["K"], s["N"], CODES[s["out"]], s["y"], s["N"], s["ws"])
    return s["y"]


PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "align": _plain_align,
         "int8": _plain_int8}
OWN = {"route": _own_route, "route_backward": _own_route_backward, "align": _own_align,
       "int8": _own_int8}


def run(s):
    if own:
        return OWN[s["op"]](s)
    return PLAIN[s["op"]](s)


# ---- definitions in 64 bits ------------------------------------------------------------
def _exact_route(c, s):
    """Expert by expert: the place of an expert is the number of experts that
    come before it (larger key, or an equal one and a lower index)."""
    x = s["x"].double()
    M, E, n = c["M"], c["E"], c["groups"]
    if c["score"] == "softmax":
        lse = torch.logsumexp(x, dim=1, keepdim=True)
        p = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse))
    else:
        p = torch.sigmoid(x)
    t = p if s["b"] is None else p + s["b"].double()
    key = x if s["b"] is None else t

    def places(v, allowed):
        """number of allowed columns before each column"""
        at = torch.zeros(v.shape, dtype=torch.int64, device=v.device)
        idx = torch.arange(v.shape[1], device=v.device)
        for j in range(v.shape[1]):
            before = (v[:, j:j + 1] > v) | ((v[:, j:j + 1] == v) & (j < idx))
            at += before & allowed[:, j:j + 1]
        return at

    allowed = torch.ones(M, E, dtype=torch.bool, device=x.device)
    if n > 1:
        if c["rule"] == "top2":
            two = t.reshape(M, n, E // n).topk(2, dim=2).values
            gs = two[:, :, 0] + two[:, :, 1]
        else:
            gs = key.reshape(M, n, E // n).max(dim=2).values
        keep = places(gs, torch.ones_like(gs, dtype=torch.bool)) < c["keep"]
        allowed = keep[:, :, None].expand(M, n, E // n).reshape(M, E)
    at = places(key, allowed)
    at = torch.where(allowed, at, E)
    ids = torch.empty(M, c["top_k"], dtype=torch.int64, device=x.device)
    for j in range(c["top_k"]):
        ids[:, j] = (at == j).int().argmax(dim=1)
    w = torch.take_along_dim(p, ids, 1)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
        w = torch.where(torch.isnan(w), 0.0, w)
    return ids.int(), w * c["scale"]


def _exact_route_backward(c, s):
    """The Jacobian's transpose, chosen expert by chosen expert."""
    x, ids, g = s["x"].double(), s["ids"].long(), s["dw"].double() * c["scale"]
    k = c["top_k"]
    p = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.sigmoid(x)
    sel = torch.stack([p[torch.arange(c["M"]), ids[:, j]] for j in range(k)], dim=1)
    if c["renorm"]:                       # w_j = s_j / S: dL/ds_j
        S = sel.sum(dim=1, keepdim=True)
        g = g / S - (g * sel).sum(dim=1, keepdim=True) / (S * S)
    ds = torch.zeros_like(x)
    for j in range(k):
        ds[torch.arange(c["M"]), ids[:, j]] += g[:, j]
    if c["score"] == "softmax":
        return p * (ds - (p * ds).sum(dim=1, keepdim=True))
    return ds * p * (1.0 - p)


def _exact_align(c, s):
    import numpy as np
    ids = s["ids"].cpu().numpy().reshape(-1).astype(np.int64) - c["first"]
    S, b, n = ids.size, c["block_m"], _padded(c)
    out = np.full(n, S, dtype=np.int32)
    labels = np.full(n // b, -1, dtype=np.int32)
    counts = np.zeros(c["E"], dtype=np.int32)
    at = 0
    for e in range(c["E"]):
        mine = np.flatnonzero(ids == e)
        counts[e] = mine.size
        out[at:at + mine.size] = mine
        blocks = -(-mine.size // b)
        labels[at // b:at // b + blocks] = e
        at += blocks * b
    return out, labels, np.array([at], dtype=np.int32), counts


def _exact_int8(c, s):
    M, N = c["M"], c["N"]
    w = s["wq"].double()
    y = torch.empty(M, N, dtype=torch.float64, device=w.device)
    for r in range(0, M, 1024):
        acc = torch.matmul(s["a"][r:r + 1024].double(), w.t())
        y[r:r + 1024] = acc * (s["sa"][r:r + 1024, None].double() * s["sw"][None].double())
    if c["bias"]:
        y += s["bias_v"].double()[None]
    if c["addend"]:
        y += s["add"].double()
    return y


def exact(c, seed):
    s = prepare(c, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward, "align": _exact_align,
            "int8": _exact_int8}[c["op"]](c, s)
