"""The general router, its gradient and the alignment of given ids on the GPU
against the float64 oracle.

Tolerances.  Weights are computed in float64 and rounded once to float32: half
a step (2^-24) and as much again for the float64 evaluation and the product
with the scale.  Gradients of chosen experts likewise, plus the half step of
the output type; the dense softmax gradient is float32 throughout (see
_dense_tol)."""

import zlib

import numpy as np
import pytest
import torch

import quantized_moe_grouped_top_amd as qm
from oracle import layer as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": (0, torch.float32), "bf16": (1, torch.bfloat16), "f16": (2, torch.float16)}


def _seed(*what):
    return zlib.crc32(repr(what).encode()) & 0x7FFFFFFF


def _logits(M, E, dtype, seed, pad=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    full = (std * torch.randn(M, E + pad, generator=g)).to(DT[dtype][1]).to(DEV)
    return full[:, :E]


def route(x, dtype, top_k, bias=None, score=0, n_group=1, topk_group=1, rule=0, renorm=True,
          scale=1.0, stream=None):
    M, E = x.shape
    ids = torch.full((M + 1, top_k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((M + 1, top_k), -7.0, device=DEV)
    qm.moe_route_topk(x, DT[dtype][0], x.stride(0) if M else E, bias, M, E, top_k, score, n_group,
                      topk_group, rule, renorm, scale, ids, w, stream=stream)
    torch.cuda.synchronize()
    assert torch.all(ids[M] == -7) and torch.all(w[M] == -7.0)    # nothing behind the last token
    return ids[:M].cpu().numpy(), w[:M].cpu().numpy()


def check_route(x, dtype, top_k, bias=None, score=0, n_group=1, topk_group=1, rule=0, renorm=True,
                scale=1.0):
    ids, w = route(x, dtype, top_k, bias, score, n_group, topk_group, rule, renorm, scale)
    ids0, w0 = L.route_general(x.float().cpu().numpy(), None if bias is None else bias.cpu().numpy(),
                               top_k, score, n_group, topk_group, rule, renorm, scale)
    assert np.array_equal(ids, ids0), np.argwhere(ids != ids0)[:4]
    fin = np.isfinite(w0)
    assert np.array_equal(fin, np.isfinite(w)) and np.array_equal(np.isnan(w0), np.isnan(w))
    err = np.abs(w[fin] - w0[fin])
    # 2^-149: below the normal range a step is absolute
    assert np.all(err <= 2.0 ** -23 * np.abs(w0[fin]) + 2.0 ** -149), err.max()


SIZES = [(1, 8, 2), (7, 8, 8), (5, 1, 1), (3, 60, 6), (64, 64, 4), (33, 96, 3), (130, 128, 8),
         (17, 160, 6), (200, 256, 8), (9, 384, 5), (65, 512, 8), (40, 511, 7), (31, 17, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,E,k", SIZES)
def test_route_plain(M, E, k, dtype):
    print(f"\n[route] plain M={M} E={E} k={k} {dtype}", flush=True)
    x = _logits(M, E, dtype, _seed(M, E, k, dtype), pad=(E * 3) % 5)
    for score in (0, 1):
        for renorm in (True, False):
            check_route(x, dtype, k, None, score, renorm=renorm, scale=1.0 + score)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,E,k", SIZES)
def test_route_bias(M, E, k, dtype):
    print(f"\n[route] bias M={M} E={E} k={k} {dtype}", flush=True)
    x = _logits(M, E, dtype, _seed(M, E, k, dtype, "b"))
    b = (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E))).to(DEV)
    for score in (0, 1):
        check_route(x, dtype, k, b, score, renorm=score == 1, scale=2.5)


@pytest.mark.parametrize("M,E,k,n,keep", [
    (1, 128, 8, 8, 4), (67, 256, 8, 8, 4), (50, 160, 6, 8, 3), (30, 60, 4, 5, 2), (21, 512, 8, 64, 9),
    (12, 96, 8, 3, 1), (9, 24, 2, 12, 1), (40, 64, 8, 16, 16), (25, 20, 4, 2, 1), (8, 128, 8, 64, 4),
    (33, 8, 2, 4, 2), (14, 384, 8, 6, 2)])
@pytest.mark.parametrize("rule", [0, 1])
def test_route_groups(M, E, k, n, keep, rule):
    print(f"\n[route] groups M={M} E={E} k={k} n={n} keep={keep} rule={rule}", flush=True)
    x = _logits(M, E, "f32", _seed(M, E, k, n, keep, rule), pad=3)
    b = (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E + n))).to(DEV)
    for score in (0, 1):
        for bias in (None, b):
            check_route(x, "f32", k, bias, score, n, keep, rule, True, 2.5)
    xb = _logits(M, E, "bf16", _seed(M, E, k, n, keep, rule, 1))
    check_route(xb, "bf16", k, b, 1, n, keep, rule, False, 1.0)


def test_route_ties_take_the_lower_expert():
    print("\n[route] ties", flush=True)
    g = torch.Generator().manual_seed(3)
    for E in (8, 16, 64, 128, 256, 512):
        x = torch.randint(-2, 3, (100, E), generator=g).float()
        x[x == 0] *= torch.where(torch.rand(int((x == 0).sum()), generator=g) < 0.5, -1.0, 1.0)
        x[0] = 0.0
        x[1] = -1.5
        x = x.to(DEV)
        b = (torch.randint(0, 2, (E,), generator=g).float() * 0.5).to(DEV)
        for score in (0, 1):
            check_route(x, "f32", 8, None, score)
            check_route(x, "f32", 8, torch.zeros(E, device=DEV), score)
            check_route(x, "f32", min(8, E // 2), None, score, 4, 2, 0)
            check_route(x, "f32", min(8, E // 2), None, score, 4, 2, 1)
        # sigmoid scores 1/2 and the bias 0 or 1/2: equal sums are exact
        check_route(torch.zeros(4, E, device=DEV), "f32", 8, b, 1, 2, 2, 1)


def test_route_masks_infinities_nan():
    print("\n[route] masks", flush=True)
    inf, nan = float("inf"), float("nan")
    for E in (8, 60, 128, 256):
        x = _logits(40, E, "f32", E).clone()
        x[:, ::3] = -inf                                          # masked experts
        x[1] = -inf                                               # nothing left
        x[2] = -inf
        x[2, E - 1] = 0.5                                         # one left
        x[3] = torch.finfo(torch.float32).min
        x[4] = -200.0                                             # sigmoid scores near 1e-87
        x[5] = -1000.0                                            # ... 0 in float64
        x[6, 1] = -torch.finfo(torch.float32).min
        x[7, 5] = 60.0
        x[8, 2] = nan
        x[9, 3], x[9, 4] = nan, nan
        x[10] = nan
        x[11, 6] = inf
        x[12, 6], x[12, 1] = inf, inf
        x[13, 6], x[13, 1] = inf, nan
        b = torch.zeros(E, device=DEV)
        b[1::4] = -inf                                            # experts out of service
        for score in (0, 1):
            for renorm in (True, False):
                check_route(x, "f32", 4, None, score, renorm=renorm)
                check_route(x, "f32", 4, None, score, 4, 2, 0, renorm)
                check_route(x[:8], "f32", 4, b, score, renorm=renorm)
                check_route(x[:8], "f32", 4, b, score, 4, 2, 1, renorm)
                check_route(x[8:], "f32", 4, b, score, renorm=renorm)
        b[0] = nan
        b[E - 1] = inf
        check_route(x[14:], "f32", 4, b, 1)
        check_route(x[14:], "f32", 2, b, 1, 2, 1, 1)


def test_route_empty_and_large():
    print("\n[route] M=0, M=70001", flush=True)
    x = torch.empty(0, 8, device=DEV)
    ids, _ = route(x, "f32", 2)
    assert ids.shape == (0, 2)
    x = _logits(70001, 128, "bf16", 9)
    b = (0.1 * torch.randn(128, generator=torch.Generator().manual_seed(1))).to(DEV)
    ids, w = route(x, "bf16", 8, b, 1, 8, 4, 1, True, 2.5)
    rows = np.r_[0:40, 35000:35040, 69961:70001]
    ids0, w0 = L.route_general(x.float().cpu().numpy()[rows], b.cpu().numpy(), 8, 1, 8, 4, 1, True, 2.5)
    assert np.array_equal(ids[rows], ids0)
    np.testing.assert_allclose(w[rows], w0, rtol=2.0 ** -23)
    assert ids.min() >= 0 and ids.max() < 128
    assert np.all(np.sort(ids, 1)[:, 1:] > np.sort(ids, 1)[:, :-1])


@pytest.mark.parametrize("M", [1500, 8200])
@pytest.mark.parametrize("E,n,keep", [(128, 8, 4), (120, 5, 2), (256, 8, 4), (250, 10, 3), (512, 16, 5)])
def test_route_many_tokens(M, E, n, keep):
    """The variants with more keys a lane, sampled rows against the oracle."""
    print(f"\n[route] many M={M} E={E}", flush=True)
    x = _logits(M, E, "f32", _seed(M, E))
    x[5, 1::2] = float("-inf")
    b = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(2))).to(DEV)
    b[::7] = float("-inf")
    rows = np.r_[0:30, M // 2:M // 2 + 20, M - 30:M]
    xs = x.cpu().numpy()[rows]
    for k in (2, 8):
        for bias, score, groups, rule in ((b, 1, n, 1), (None, 0, 1, 0), (b, 0, n, 0), (None, 1, n, 1)):
            ids, w = route(x, "f32", k, bias, score, groups, keep if groups > 1 else 1, rule, True, 2.5)
            ids0, w0 = L.route_general(xs, None if bias is None else b.cpu().numpy(), k, score, groups,
                                       keep if groups > 1 else 1, rule, True, 2.5)
            assert np.array_equal(ids[rows], ids0)
            assert np.all(np.abs(w[rows] - w0) <= 2.0 ** -23 * w0)


@pytest.mark.parametrize("E,n,keep", [(160, 8, 3), (150, 5, 2), (192, 8, 4), (176, 2, 1), (200, 8, 3),
                                      (256, 32, 8), (320, 16, 4), (300, 5, 2), (384, 8, 3), (370, 37, 9),
                                      (130, 10, 3)])
def test_route_many_tokens_of_odd_numbers_of_experts(E, n, keep):
    """20 and 24 keys a lane, groups of whole lanes and others."""
    M = 8200
    print(f"\n[route] many M={M} E={E}", flush=True)
    for dtype, pad in (("f32", 0), ("bf16", 0), ("f16", 3)):
        x = _logits(M, E, dtype, _seed(M, E, dtype), pad=pad)
        x[M - 3, 1::2] = float("-inf")
        b = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(3))).to(DEV)
        rows = np.r_[0:20, M // 2:M // 2 + 20, M - 20:M]
        xs = x.float().cpu().numpy()[rows]
        for k in (2, 8):
            for bias, score, groups, rule, renorm in ((b, 1, n, 1, True), (None, 0, 1, 0, False),
                                                      (b, 0, n, 0, False), (None, 1, n, 1, True)):
                ids, w = route(x, dtype, k, bias, score, groups, keep if groups > 1 else 1, rule, renorm, 2.5)
                ids0, w0 = L.route_general(xs, None if bias is None else b.cpu().numpy(), k, score, groups,
                                           keep if groups > 1 else 1, rule, renorm, 2.5)
                assert np.array_equal(ids[rows], ids0)
                assert np.all(np.abs(w[rows] - w0) <= 2.0 ** -23 * w0)


# ---- masked experts beside a bias, scores that are no numbers -------------------------
@pytest.mark.parametrize("M", [40, 8200])
@pytest.mark.parametrize("E,n,keep,k", [(8, 2, 1, 2), (60, 5, 2, 4), (128, 8, 4, 8), (160, 8, 3, 6),
                                        (250, 10, 3, 8), (512, 16, 5, 8)])
def test_route_masked_logits_beside_a_bias(M, E, n, keep, k):
    """A -inf logit takes its expert out whatever its bias: the choice is the one
    of the same router without these experts (their softmax terms are exp(-inf) =
    0).  Both lists of weights are within 2^-23 of the same exact values."""
    print(f"\n[route] masked beside a bias M={M} E={E}", flush=True)
    gs = E // n
    gone = np.sort(np.concatenate([g * gs + np.arange(1, gs // 2 + 1) % gs for g in range(n)]))
    left = np.setdiff1d(np.arange(E), gone)
    x = _logits(M, E, "f32", _seed(M, E, "gone"))
    x[:, left[0]] = -90.0                                         # a sigmoid score near 1e-39
    x[:, gone] = float("-inf")
    b = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    b[gone] = 0.9                                                 # what a balance bias grows to
    zero = torch.zeros(E)
    xl = x[:, left].contiguous()
    few = np.r_[0:30, M - 10:M]
    for bias in (b, zero):
        bd, bl = bias.to(DEV), bias[left].contiguous().to(DEV)
        for score in (0, 1):
            for groups, rule in ((1, 0), (n, 0), (n, 1)):
                if rule == 1 and left.size // n < 2:
                    continue
                got, w = route(x, "f32", k, bd, score, groups, keep if groups > 1 else 1, rule, True, 2.5)
                assert not np.isin(got, gone).any(), (score, groups, rule)
                want, w0 = route(xl, "f32", k, bl, score, groups, keep if groups > 1 else 1, rule, True, 2.5)
                assert np.array_equal(got, left[want]), (score, groups, rule)
                assert np.all(np.abs(w.astype(np.float64) - w0) <= 2.0 ** -22 * w0)
                ids0, _ = L.route_general(x.cpu().numpy()[few], bias.numpy(), k, score, groups,
                                          keep if groups > 1 else 1, rule, True, 2.5)
                assert np.array_equal(got[few], ids0)


def test_route_fewer_experts_left_than_choices_beside_a_bias():
    """Masked experts follow the others, lower expert first, with weight 0."""
    print("\n[route] few left beside a bias", flush=True)
    for E in (8, 64, 256):
        x = torch.full((3, E), float("-inf"))
        x[1, E - 1] = -95.0
        x[2, 2], x[2, E - 2] = 0.25, -1.0
        b = torch.linspace(-1.0, 1.0, E)
        for score in (0, 1):
            ids, w = route(x.to(DEV), "f32", 4, b.to(DEV), score, renorm=False)
            assert list(ids[0]) == [0, 1, 2, 3] and list(ids[1]) == [E - 1, 0, 1, 2]
            assert list(ids[2]) in ([2, E - 2, 0, 1], [E - 2, 2, 0, 1])
            assert np.all(w[0] == 0) and np.all(w[1:, 2:] == 0) and np.all(w[2, :2] > 0)
            check_route(x.to(DEV), "f32", 4, b.to(DEV), score)


@pytest.mark.parametrize("M", [24, 8200])
def test_route_softmax_with_a_nan_that_is_not_chosen(M):
    """A NaN or +inf logit makes every softmax score of its token NaN, the
    renormalised weights of other experts too; other tokens keep theirs."""
    print(f"\n[route] NaN M={M}", flush=True)
    for E in (16, 60, 128, 256, 512):
        x = _logits(M, E, "f32", _seed(M, E, "nan"))
        x[3, E - 6] = float("nan")
        x[5, E - 5] = float("inf")
        x[7, E - 6], x[7, E - 5] = float("nan"), float("-inf")
        bad = [3, 5, 7]
        fine = np.setdiff1d(np.arange(M), bad)
        for bias, groups, rule in ((torch.zeros(E, device=DEV), 1, 0), (None, 4, 1),
                                   (torch.zeros(E, device=DEV), 4, 1)):
            for renorm in (True, False):
                ids, w = route(x, "f32", 4, bias, 0, groups, max(1, groups // 2), rule, renorm, 1.5)
                assert np.all(np.isnan(w[bad])) and np.all(np.isfinite(w[fine])), (E, groups, renorm)
                assert np.all((ids >= 0) & (ids < E))
                check_route(x[:24], "f32", 4, bias, 0, groups, max(1, groups // 2), rule, renorm, 1.5)


# ---- gradient ----------------------------------------------------------------------
def _dense_tol(x, ids, g, scale):
    """Bound for the dense softmax gradient in float32.  p = exp(x - m) / Z:
    the rounded difference x - m carries |x - m| 2^-24 into exp, exp and the
    division a few half steps, the sum over E values in pieces of at most 16
    and a tree over 64 lanes 24 of them; u and the difference g - u add as many
    relative to |g| + sum |g_i| p_i."""
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        d = np.max(x, 1, keepdims=True) - x
    p = np.stack([L._softmax(r) for r in x])
    up = np.zeros_like(x)
    total = np.zeros((x.shape[0], 1))
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if 0 <= e < x.shape[1]:
                up[t, e] += abs(g[t, j])
                total[t] += abs(g[t, j]) * p[t, e]
    d = np.where(np.isfinite(d), d, 0.0)
    spread = np.max(np.where(p > 1e-12, d, 0.0), 1, keepdims=True)
    return scale * p * (up + total) * 2.0 ** -24 * (d + spread + 64)


def check_backward(x, dtype, ids, g, score, renorm, scale, pad=0, ref=None):
    M, E = x.shape
    k = ids.shape[1]
    full = torch.full((M + 1, E + pad), 77.0, dtype=DT[dtype][1], device=DEV)
    qm.moe_route_topk_backward(g, ids, x, DT[dtype][0], x.stride(0), M, E, k, score, renorm, scale,
                               full, E + pad)
    torch.cuda.synchronize()
    assert torch.all(full[M] == 77.0) and torch.all(full[:, E:] == 77.0)
    got = full[:M, :E].double().cpu().numpy()
    gs = (g if ref is None else ref).cpu().numpy()
    xs, cs = x.float().cpu().numpy(), ids.cpu().numpy()
    ref = L.route_backward(gs, cs, xs, score, renorm, scale)
    eps = torch.finfo(DT[dtype][1]).eps / 2
    tiny = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dtype]
    mag = scale * np.abs(gs).max() if gs.size else 0.0
    tol = (eps + 2.0 ** -23) * np.abs(ref) + tiny + 2.0 ** -48 * mag * k
    if score == 0 and not renorm:
        tol = tol + _dense_tol(xs, cs, gs, scale)
    # an expert chosen more than once: its at most k shares, each at most 2 mag
    # (a share is scale * s * (g - u) with s <= 1 and |u| <= max|g|), are rounded
    # to float32 (half a step each) and added in float32 (half a step of the
    # partial sum each): 2^-24 * (2 mag k + 2 mag k)
    for t in range(M):
        ids_t, n = np.unique(cs[t][(cs[t] >= 0) & (cs[t] < E)], return_counts=True)
        tol[t, ids_t[n > 1]] += 2.0 ** -24 * 4 * mag * k
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])
    outside = np.ones((M, E), bool)
    for t in range(M):
        outside[t, cs[t][(cs[t] >= 0) & (cs[t] < E)]] = False
    if not (score == 0 and not renorm):
        assert np.all(got[outside] == 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,E,k", SIZES)
def test_route_backward(M, E, k, dtype):
    print(f"\n[route backward] M={M} E={E} k={k} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(_seed(M, E, k))
    x = _logits(M, E, dtype, _seed(M, E, k, dtype, "g"), pad=(E * 3) % 5)
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(M)]).int().to(DEV)
    g = torch.randn(M, k, generator=gen).to(DEV)
    for score in (0, 1):
        for renorm in (True, False):
            check_backward(x, dtype, ids, g, score, renorm, 2.5, pad=E % 3)


def test_route_backward_odd_choices_and_masks():
    print("\n[route backward] odd choices, masks", flush=True)
    inf = float("inf")
    x = _logits(12, 32, "f32", 5).clone()
    gen = torch.Generator().manual_seed(2)
    ids = torch.stack([torch.randperm(32, generator=gen)[:4] for _ in range(12)]).int()
    ids[0, 1] = ids[0, 0]                                          # the same expert twice
    ids[1] = 7                                                     # ... four times
    ids[2, 2] = -1                                                 # dropped
    ids[3] = -1                                                    # all dropped
    ids[4, 0], ids[4, 3] = 32, 1 << 30                             # beyond the experts
    x[5, ids[5, 0].item()] = -inf
    x[6] = -inf
    x[7] = -300.0                                                  # sigmoid scores near 1e-131
    x[8] = 90.0
    x[9, ids[9].long()] = -inf                                     # all chosen masked
    g = torch.randn(12, 4, generator=gen)
    g[2, 2], g[3, 0], g[4, 0] = float("nan"), inf, float("nan")    # of choices that take no part
    ref = torch.where(torch.isfinite(g), g, 0.0)
    for score in (0, 1):
        for renorm in (True, False):
            check_backward(x, "f32", ids.to(DEV), g.to(DEV), score, renorm, 1.5, pad=1, ref=ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route_backward_of_the_largest_and_lowest_values(dtype):
    """Rows masked with their type's lowest value, whole rows among them: all
    logits are equal there, so every softmax score is 1 / E."""
    print(f"\n[route backward] largest and lowest {dtype}", flush=True)
    lowest = torch.finfo(DT[dtype][1]).min
    for E, k in ((24, 4), (128, 8), (300, 5)):
        gen = torch.Generator().manual_seed(E)
        x = _logits(7, E, dtype, E).clone()
        x[0] = lowest
        x[1] = -lowest
        x[2, ::2] = lowest
        x[3] = lowest
        x[3, 1] = -lowest                                          # one takes all
        x[4, 3:] = -lowest                                         # E - 3 share
        x[5, :] = lowest
        x[5, 2] = 0.0
        ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(7)]).int().to(DEV)
        g = torch.randn(7, k, generator=gen).to(DEV)
        for score in (0, 1):
            for renorm in (True, False):
                check_backward(x, dtype, ids, g, score, renorm, 1.5)


@pytest.mark.parametrize("score,renorm", [(0, False), (0, True), (1, False), (1, True)])
def test_route_backward_in_place(score, renorm):
    print("\n[route backward] in place", flush=True)
    for M, E, dtype in ((1, 8, "f32"), (333, 60, "bf16"), (2000, 256, "f32"), (70, 512, "f16")):
        gen = torch.Generator().manual_seed(E)
        x = _logits(M, E, dtype, E + 1, pad=8)
        ids = torch.stack([torch.randperm(E, generator=gen)[:8] for _ in range(M)]).int().to(DEV)
        g = torch.randn(M, 8, generator=gen).to(DEV)
        dx = torch.empty(M, E + 8, dtype=x.dtype, device=DEV)
        for d in (dx, x):
            qm.moe_route_topk_backward(g, ids, x, DT[dtype][0], E + 8, M, E, 8, score, renorm, 2.0, d, E + 8)
        torch.cuda.synchronize()
        assert torch.equal(dx[:, :E], x)


def test_route_backward_against_differences():
    """The gradient of the kernel's own weights: sum_j g_j w_j by central
    differences.  The weights are float32 (half a step of 2^-24 of up to 1 on
    each side), so a step of 2^-6 leaves 8 * 2^-24 * 2^6 = 2^-15 of noise and
    h^2 |f'''| / 6 < 2^-12 * |g| of curvature (f''' of scores below 1)."""
    print("\n[route backward] differences", flush=True)
    gen = torch.Generator().manual_seed(4)
    E, k, h = 16, 4, 2.0 ** -6
    x = torch.randn(1, E, generator=gen)
    order = x.argsort(dim=1, descending=True)
    x[0, order[0]] = torch.linspace(1.5, -1.5, E)                  # gaps well above h
    g = torch.randn(1, k, generator=gen)
    for score in (0, 1):
        for renorm in (True, False):
            ids, _ = route(x.to(DEV), "f32", k, None, score, renorm=renorm)
            dx = torch.empty(1, E, device=DEV)
            qm.moe_route_topk_backward(g.to(DEV), torch.from_numpy(ids).to(DEV), x.to(DEV), 0, E, 1,
                                       E, k, score, renorm, 1.0, dx, E)
            both = x.repeat(2 * E, 1)
            for e in range(E):
                both[2 * e, e] += h
                both[2 * e + 1, e] -= h
            ids2, w2 = route(both.to(DEV), "f32", k, None, score, renorm=renorm)
            assert np.all(ids2 == ids)
            f = (w2.astype(np.float64) * g.numpy()).sum(1)
            diff = (f[0::2] - f[1::2]) / (2 * h)
            assert np.abs(diff - dx.cpu().numpy()[0]).max() < 2.0 ** -15 + 2.0 ** -12 * g.abs().max().item()


# ---- the plain softmax gradient of confident tokens -----------------------------------
def _dense_reference(x, ids, g, scale):
    """Plain softmax gradient of one token in float64 without the difference of
    nearly equal terms, dx_e = scale p_e (g_e sum_{i != e} p_i - sum_{i != e} g_i p_i),
    and a bound for its evaluation in float32 in this form.  In half steps
    (2^-24): x - m carries |x - m| of them into the exponential, its product with
    log2(e) and that constant 1.5 |x - m|, the exponential 2; sums are pieces
    of at most 24 and a tree over 64 lanes, at most 30; the division 3; z minus the
    own term doubles what z carries; products, scale and differences one each: at
    most 128 without the exponentials."""
    x, g = x.astype(np.float64), g.astype(np.float64)
    E = x.size
    d = x.max() - x
    p = np.exp(-d)
    p /= p.sum()
    up, mag = np.zeros(E), np.zeros(E)
    for j, e in enumerate(ids):
        if 0 <= e < E:
            up[e] += g[j]
            mag[e] += abs(g[j])
    own = 2.5 * d + 2
    out, tol = np.empty(E), np.empty(E)
    for e in range(E):
        o = np.arange(E) != e
        out[e] = scale * p[e] * (up[e] * p[o].sum() - (up[o] * p[o]).sum())
        terms = (mag[e] + mag[o]) * p[o]
        tol[e] = scale * p[e] * 2.0 ** -24 * ((128 + own[e]) * terms.sum() + (own[o] * terms).sum())
    return out, tol


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,k", [(8, 8), (24, 3), (60, 6), (128, 8), (200, 8), (256, 8), (512, 8)])
def test_route_backward_of_confident_tokens(E, k, dtype):
    """One logit 0 to 30 above the others, chosen in most tokens: its gradient is
    a small difference of large terms, and holds relative to what is left."""
    print(f"\n[route backward] confident E={E} k={k} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(_seed(E, k, dtype))
    M = 32
    x = 0.25 * torch.randn(M, E, generator=gen)
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(M)]).int()
    for t in range(M):
        x[t, ids[t, t % k]] = float(t)                            # the t-th token's gap, nearly
    x[9, ids[9, 0]] = x[9, ids[9, 1]] = 12.0                      # two share the maximum
    x[10] = -3.0
    x[10, (int(ids[10].max()) + 1) % E] = 14.0                    # perhaps not chosen
    ids[11, 1] = ids[11, 11 % k]                                  # the maximum twice
    ids[12, (12 % k + 1) % k] = -1
    x = x.to(DT[dtype][1])
    g = torch.randn(M, k, generator=gen)
    dx = torch.empty(M, E, dtype=DT[dtype][1], device=DEV)
    qm.moe_route_topk_backward(g.to(DEV), ids.to(DEV), x.to(DEV), DT[dtype][0], E, M, E, k, 0, False, 2.5,
                               dx, E)
    torch.cuda.synchronize()
    got = dx.double().cpu().numpy()
    tiny = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}[dtype]
    eps = torch.finfo(DT[dtype][1]).eps / 2
    for t in range(M):
        ref, tol = _dense_reference(x[t].double().numpy(), ids[t].numpy(), g[t].numpy(), 2.5)
        tol = tol + eps * (np.abs(ref) + tol) + tiny
        bad = np.abs(got[t] - ref) > tol
        assert not bad.any(), (t, np.argwhere(bad)[:3], got[t][bad][:3], ref[bad][:3], tol[bad][:3])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,k", [(8, 8), (60, 3), (128, 8), (512, 2)])
def test_route_backward_of_confident_renormalised_tokens(E, k, dtype):
    """Renormalised weights of which one is nearly 1.  dx_j = scale ds_j/dx_j (g_j
    sum_{i != j} s_i - sum_{i != j} g_i s_i) / S^2 has no difference of nearly
    equal terms; in float64 it holds to 2^-45 of the terms' magnitude
    (some ten roundings of 2^-53, the exponentials included), then the result is
    rounded to float32 and to its type."""
    print(f"\n[route backward] confident, renormalised E={E} k={k} {dtype}", flush=True)
    gen = torch.Generator().manual_seed(_seed(E, k, dtype, "renorm"))
    M = 40
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(M)]).int()
    g = torch.randn(M, k, generator=gen)
    eps = torch.finfo(DT[dtype][1]).eps / 2 + 2.0 ** -24
    tiny = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}[dtype]
    for score in (0, 1):
        x = 0.25 * torch.randn(M, E, generator=gen) - (6.0 if score else 0.0)
        for t in range(M):                                        # gaps from 0 to 39
            x[t, ids[t, t % k]] = float(t) if score == 0 else 2.0
            if score:
                x[t, ids[t][torch.arange(k) != t % k].long()] -= float(t) - 8.0
        x = x.to(DT[dtype][1])
        dx = torch.empty(M, E, dtype=DT[dtype][1], device=DEV)
        qm.moe_route_topk_backward(g.to(DEV), ids.to(DEV), x.to(DEV), DT[dtype][0], E, M, E, k, score, True,
                                   2.5, dx, E)
        torch.cuda.synchronize()
        got = np.take_along_axis(dx.double().cpu().numpy(), ids.numpy().astype(np.int64), 1)
        v = np.take_along_axis(x.double().numpy(), ids.numpy().astype(np.int64), 1)
        gd = g.double().numpy()
        for t in range(M):
            s = np.exp(v[t] - v[t].max()) if score == 0 else 1.0 / (1.0 + np.exp(-v[t]))
            slope = s if score == 0 else s / (1.0 + np.exp(v[t]))
            for j in range(k):
                o = np.arange(k) != j
                c = 2.5 * slope[j] / s.sum() ** 2
                ref = c * ((gd[t, j] - gd[t, o]) * s[o]).sum()
                mag = c * ((abs(gd[t, j]) + abs(gd[t, o])) * s[o]).sum()
                assert abs(got[t, j] - ref) <= eps * abs(ref) + 2.0 ** -45 * mag + tiny, (score, t, j)


def test_route_backward_of_sigmoid_scores_near_the_smallest_float64():
    """Equal logits down to -745, where a score is the smallest float64: every choice
    has 1 / k of their sum.  (exp(-x) alone overflows below -709.)"""
    print("\n[route backward] smallest scores", flush=True)
    g = torch.randn(4, 4, generator=torch.Generator().manual_seed(8))
    x = torch.tensor([-700.0, -715.0, -740.0, -60000.0])[:, None].repeat(1, 16)
    ids = torch.tensor([[3, 0, 15, 7]]).repeat(4, 1).int()
    dx = torch.empty(4, 16, device=DEV)
    qm.moe_route_topk_backward(g.to(DEV), ids.to(DEV), x.to(DEV), 0, 16, 4, 16, 4, 1, True, 1.5, dx, 16)
    torch.cuda.synchronize()
    gd = g.double()
    want = torch.zeros(4, 16, dtype=torch.float64)
    want[:3].scatter_(1, ids[:3].long(), 1.5 * 0.25 * (gd - gd.mean(1, keepdim=True))[:3])
    # three roundings of 2^-53 and those to float32
    assert torch.all((dx.cpu().double() - want).abs() <= 2.0 ** -23 * want.abs() + 2.0 ** -48)
    got, w = route(x.to(DEV), "f32", 4, None, 1, renorm=True, scale=1.5)
    assert np.all(got == np.arange(4)) and np.all(w[:3] == np.float32(0.375)) and np.all(w[3] == 0)
    check_route(x.to(DEV), "f32", 4, None, 1)
    check_backward(x[:2].to(DEV), "f32", ids[:2].to(DEV), g[:2].to(DEV), 1, True, 1.5)


# ---- alignment ------------------------------------------------------------------------
def check_align(ids, E, block_m, first=0, counts=True):
    M, k = ids.shape
    n = qm.moe_align_max_padded(M, E, k, block_m)
    dev = torch.from_numpy(np.ascontiguousarray(ids)).to(DEV)
    s = torch.full((n + 1,), -9, dtype=torch.int32, device=DEV)
    e = torch.full((n // block_m + 1,), -9, dtype=torch.int32, device=DEV)
    p = torch.full((2,), -9, dtype=torch.int32, device=DEV)
    c = torch.full((E + 1,), -9, dtype=torch.int32, device=DEV) if counts else None
    wb = qm.moe_align_workspace_bytes(M, E, k)
    ws = torch.full((wb // 4 + 1,), 0x3fffffff, dtype=torch.int32, device=DEV)
    qm.moe_align_topk_ids(dev, M, E, k, block_m, first, s, e, p, c, ws)
    torch.cuda.synchronize()
    s0, e0, p0, c0 = L.align_ids(ids, E, block_m, first)
    np.testing.assert_array_equal(s[:-1].cpu().numpy(), s0)
    np.testing.assert_array_equal(e[:-1].cpu().numpy(), e0)
    assert p[0].item() == p0
    assert s[-1] == -9 and e[-1] == -9 and p[1] == -9 and ws[-1] == 0x3fffffff
    if counts:
        np.testing.assert_array_equal(c[:-1].cpu().numpy(), c0)
        assert c[-1] == -9


@pytest.mark.parametrize("M,E,k,bm", [
    (1, 1, 1, 16), (1, 8, 2, 128), (64, 8, 2, 16), (37, 60, 6, 32), (511, 128, 2, 64), (512, 64, 2, 16),
    (513, 128, 2, 256), (1000, 128, 8, 128), (3000, 96, 5, 16), (8192, 128, 8, 128),
    (65536, 1, 1, 16), (8191, 8, 8, 64), (4096, 3, 2, 128)])
def test_align_ids(M, E, k, bm):
    print(f"\n[align ids] M={M} E={E} k={k} block_m={bm}", flush=True)
    rng = np.random.default_rng(M + E)
    x = rng.standard_normal((M, E)) + rng.standard_normal(E)
    ids = np.argsort(-x, axis=1)[:, :k].astype(np.int32)
    check_align(ids, E, bm)
    check_align(ids, E, bm, counts=False)
    if E >= 4:
        lo = E // 3                                              # a window of local experts
        if k <= E - lo - 1:
            check_align(ids, E - lo - 1, bm, first=lo)


def test_align_ids_dropped_and_skewed():
    print("\n[align ids] dropped, skewed", flush=True)
    rng = np.random.default_rng(0)
    check_align(np.full((40, 2), -1, np.int32), 8, 16)              # nothing stays
    check_align(np.full((5000, 2), 7, np.int32), 8, 16)             # one expert takes all
    check_align(np.full((8192, 8), 127, np.int32), 128, 128)
    ids = rng.integers(-4, 12, (3000, 4)).astype(np.int32)
    ids[5] = [2147483647, -2147483648, 0, 7]
    check_align(ids, 8, 32)
    check_align(ids, 8, 32, first=-2147483648)
    check_align(ids, 8, 32, first=2147483640)
    check_align(np.zeros((0, 2), np.int32), 8, 16)                  # no tokens: buffers written


def test_align_ids_equals_the_fused_alignment():
    """Routed by the fused call, its ids aligned again: the same buffers."""
    print("\n[align ids] against moe_align_block_size", flush=True)
    for M, E, k, bm in [(64, 8, 2, 16), (3000, 64, 4, 128)]:
        x = _logits(M, E, "f32", M)
        n = qm.moe_align_max_padded(M, E, k, bm)
        new = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        ids, s, e, p = new(M, k), new(n), new(n // bm), new(1)
        w = torch.empty(M, k, device=DEV)
        qm.moe_align_block_size(x, M, E, k, bm, ids, w, s, e, p)
        s2, e2, p2 = new(n), new(n // bm), new(1)
        ws = new(qm.moe_align_workspace_bytes(M, E, k) // 4)
        qm.moe_align_topk_ids(ids, M, E, k, bm, 0, s2, e2, p2, None, ws)
        ids2, w2 = route(x, "f32", k)
        torch.cuda.synchronize()
        assert torch.equal(s, s2) and torch.equal(e, e2) and torch.equal(p, p2)
        assert np.array_equal(ids.cpu().numpy(), ids2)
        np.testing.assert_allclose(w.cpu().numpy(), w2, rtol=1e-6)
