"""The operators around the grouped GEMMs without a GPU: exports, sizes, every
refusal (before anything is enqueued), and the oracle they are tested
against: brute force, closed forms and central differences."""

import ctypes
import os
import re

import numpy as np
import pytest

import quantized_moe_grouped_top_amd as qm
from oracle import layer as L
from oracle import moe as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_layer.h")
FAKE = 1 << 20
INV, UNS = qm.MOE_EINVAL, qm.MOE_EUNSUPPORTED


def _gpu_visible():
    import torch
    return torch.cuda.is_available()


needs_lib = pytest.mark.skipif(not os.path.exists(qm.LIB_PATH), reason="libqmoe.so not built")
no_gpu = pytest.mark.skipif(_gpu_visible(), reason="fake-pointer error paths run only without a GPU")


@needs_lib
def test_layer_symbols():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(qm.LAYER_EXPORTS)
    h = ctypes.CDLL(qm.LIB_PATH)
    for n in names:
        assert hasattr(h, n), n


@needs_lib
def test_layer_sizes():
    assert qm.moe_align_workspace_bytes(64, 8, 2) == 8 * 4
    assert qm.moe_align_workspace_bytes(8192, 128, 8) == 64 * 128 * 4
    assert qm.moe_align_workspace_bytes(0, 8, 2) == 0
    assert qm.moe_align_workspace_bytes(64, 200, 2) == 0
    for M, K, N in [(1, 1, 1), (1, 14336, 64), (64, 4096, 14336), (4096, 14336, 4096),
                    (512, 131071, 64), (4096, 131071, 4096)]:
        assert 0 <= qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N) <= 64 << 20
    assert qm.moe_gemm_int8w8a8_workspace_bytes(0, 64, 64) == 0
    assert qm.moe_gemm_int8w8a8_workspace_bytes(4, 1 << 20, 64) == 0


@needs_lib
def test_int8_workspace_holds_the_shares_and_is_at_most_16_mib():
    """One int32 sum of every output and share, columns padded to four: a share of 2048 k
    at least in 16-row tiles (14336 / 2048 = 7), 256 CUs over 64 tiles of 64 x 16, all
    shares of a XCD's 128 x 128 tiles on its 32 CUs (16 tiles: 2), at most 16; 256
    tiles of 128 x 128 are 2^24 bytes."""
    for M, K, N, shares in [(1, 14336, 64, 7), (64, 14336, 1024, 4), (512, 14336, 4096, 2),
                            (512, 131071, 130, 16), (4096, 14336, 4096, 0), (16, 64, 16, 0), (1, 15, 4096, 0)]:
        assert qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N) == shares * M * ((N + 3) // 4 * 4) * 4, (M, K, N)
    rng = np.random.default_rng(0)
    for _ in range(4000):
        M, K, N = (int(2.0 ** v) for v in rng.uniform((0, 0, 0), (18, 16.99, 18)))
        n = qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N)
        assert 0 <= n <= 16 << 20 and n % (M * ((N + 3) // 4 * 4) * 4) == 0, (M, K, N)


def _route(**kw):
    a = dict(logits=FAKE, dtype=0, ld=128, bias=FAKE, M=16, E=128, top_k=8, score=1, n_group=8,
             topk_group=4, group_rule=1, renormalize=1, scale=2.5, topk_ids=FAKE,
             topk_weights=FAKE, stream=0)
    a.update(kw)
    return qm.moe_route_topk(**a)


@needs_lib
@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), INV), (dict(score=2), INV), (dict(group_rule=2), INV), (dict(M=-1), INV),
    (dict(E=0), INV), (dict(E=513, ld=600, n_group=1, topk_group=1), UNS),
    (dict(top_k=0), INV), (dict(top_k=129), INV), (dict(top_k=9), UNS), (dict(ld=127), INV),
    (dict(ld=1 << 31), UNS), (dict(n_group=7), INV), (dict(n_group=0), INV),
    (dict(n_group=128), UNS), (dict(topk_group=0), INV), (dict(topk_group=9), INV),
    (dict(n_group=32, topk_group=1), INV),                       # 4 experts for 8 choices
    (dict(E=8, ld=8, top_k=2, n_group=8, topk_group=4), INV),     # two best of one expert
    (dict(logits=0), INV), (dict(topk_ids=None), INV), (dict(topk_weights=0), INV),
    (dict(logits=FAKE + 2), INV), (dict(bias=FAKE + 1), INV), (dict(topk_ids=FAKE + 2), INV),
    (dict(dtype=1, logits=FAKE + 1), INV), (dict(M=1 << 25), UNS),
])
def test_route_rejects(kw, code):
    with pytest.raises(qm.MoeError) as ei:
        _route(**kw)
    assert ei.value.code == code and "moe_route_topk" in str(ei.value)


def _bwd(**kw):
    a = dict(d_weights=FAKE, topk_ids=FAKE, logits=FAKE, dtype=0, ld=64, M=16, E=64, top_k=4,
             score=0, renormalize=1, scale=1.0, d_logits=FAKE, ldd=64, stream=0)
    a.update(kw)
    return qm.moe_route_topk_backward(**a)


@needs_lib
@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), INV), (dict(score=5), INV), (dict(E=600, ld=600, ldd=600), UNS),
    (dict(top_k=65), INV), (dict(top_k=9), UNS), (dict(ld=63), INV), (dict(ldd=63), INV),
    (dict(ldd=1 << 31), UNS), (dict(d_weights=0), INV), (dict(topk_ids=0), INV),
    (dict(logits=0), INV), (dict(d_logits=0), INV), (dict(d_logits=FAKE + 2), INV),
    (dict(d_weights=FAKE + 2), INV), (dict(M=-2), INV),
])
def test_route_backward_rejects(kw, code):
    with pytest.raises(qm.MoeError) as ei:
        _bwd(**kw)
    assert ei.value.code == code


def _align(**kw):
    a = dict(topk_ids=FAKE, M=64, E=8, top_k=2, block_m=16, expert_first=0, sorted_token_ids=FAKE,
             expert_ids=FAKE, num_tokens_post_padded=FAKE, expert_counts=None, workspace=FAKE,
             stream=0)
    a.update(kw)
    return qm.moe_align_topk_ids(**a)


@needs_lib
@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(E=129), INV), (dict(E=0), INV), (dict(top_k=9, E=16), UNS), (dict(top_k=9), INV),
    (dict(M=-1), INV), (dict(M=40000), UNS), (dict(block_m=24), UNS), (dict(topk_ids=0), INV),
    (dict(sorted_token_ids=0), INV), (dict(expert_ids=0), INV),
    (dict(num_tokens_post_padded=0), INV), (dict(workspace=None), INV),
    (dict(workspace=FAKE + 2), INV), (dict(topk_ids=FAKE + 1), INV),
    (dict(expert_counts=FAKE + 2), INV),
])
def test_align_ids_rejects(kw, code):
    with pytest.raises(qm.MoeError) as ei:
        _align(**kw)
    assert ei.value.code == code


@needs_lib
@no_gpu
@pytest.mark.parametrize("M,E,top_k", [(8193, 128, 8), (65537, 8, 1), (2147483647, 128, 8), (64, 8, 9),
                                       (64, 2, 4), (-1, 8, 2), (64, 0, 1), (64, 129, 2), (64, 8, 0)])
def test_align_workspace_of_refused_sizes_is_0(M, E, top_k):
    with pytest.raises(qm.MoeError):
        _align(M=M, E=E, top_k=top_k)
    assert qm.moe_align_workspace_bytes(M, E, top_k) == 0


def _int8(**kw):
    a = dict(a_q=FAKE, lda=64, a_scale=FAKE, w_q=FAKE, ldw=64, w_scale=FAKE, bias=None,
             addend=None, M=4, K=64, N=32, out_dtype=1, out=FAKE, ldo=32, workspace=None, stream=0)
    a.update(kw)
    return qm.moe_gemm_int8w8a8(**a)


@needs_lib
@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(out_dtype=3), INV), (dict(M=-1), INV), (dict(K=0), INV), (dict(N=0), INV),
    (dict(K=131072, lda=131072, ldw=131072), UNS), (dict(lda=63), INV), (dict(ldw=63), INV),
    (dict(ldo=31), INV), (dict(lda=1 << 22), UNS), (dict(ldw=1 << 22), UNS),
    (dict(ldo=1 << 22), UNS), (dict(a_q=0), INV), (dict(a_scale=0), INV), (dict(w_q=0), INV),
    (dict(w_scale=0), INV), (dict(out=0), INV), (dict(out=FAKE + 1), INV),
    (dict(out_dtype=0, out=FAKE + 2), INV), (dict(addend=FAKE + 1), INV),
    (dict(bias=FAKE + 2), INV), (dict(a_scale=FAKE + 1), INV), (dict(workspace=FAKE + 8), INV),
])
def test_int8_rejects(kw, code):
    with pytest.raises(qm.MoeError) as ei:
        _int8(**kw)
    assert ei.value.code == code


@needs_lib
@no_gpu
@pytest.mark.parametrize("kw", [
    dict(M=1 << 27), dict(M=2147483647), dict(N=1 << 22, ldo=1 << 22),
    dict(M=1 << 26, N=1 << 10, ldo=1 << 10), dict(M=(1 << 27) - 1, N=513, ldo=513)])
def test_int8_rejects_more_than_one_launch_holds(kw):
    with pytest.raises(qm.MoeError) as ei:
        _int8(**kw)
    assert ei.value.code == UNS
    sizes = dict(M=16, K=64, N=32)
    sizes.update({k: v for k, v in kw.items() if k in sizes})
    assert qm.moe_gemm_int8w8a8_workspace_bytes(**sizes) == 0


@needs_lib
@no_gpu
def test_runner_classes_refuse_other_shapes_and_types():
    import torch
    from quantized_moe_grouped_top_amd import runner
    r = runner.TopKRouter(4, 8, 2, device="cpu")
    x, g = torch.zeros(4, 8), torch.zeros(4, 2)
    for call in (lambda: r.route(x.double()), lambda: r.route(x[:3]), lambda: r.route(x.t()),
                 lambda: r.route(x, torch.zeros(7)), lambda: r.route(x, torch.zeros(8).double()),
                 lambda: r.backward(torch.zeros(2, 4).t(), x), lambda: r.backward(g.double(), x),
                 lambda: r.backward(g, x[:3])):
        with pytest.raises(AssertionError):
            call()
    lin = runner.Int8Linear(4, 32, 16, device="cpu")
    w, s = torch.zeros(16, 32, dtype=torch.int8), torch.zeros(16)
    out = torch.zeros(4, 16, dtype=torch.bfloat16)
    for call in (lambda: lin.gemm(w.t(), s), lambda: lin.gemm(w[:8], s), lambda: lin.gemm(w, s[:8]),
                 lambda: lin.gemm(w, s, bias=torch.zeros(8)), lambda: lin.gemm(w, s, out=out.float()),
                 lambda: lin.gemm(w, s, addend=out[:, :8]), lambda: lin.gemm(w, s, addend=out[:2])):
        with pytest.raises(AssertionError):
            call()


@needs_lib
@no_gpu
def test_linear_quantizes_only_its_own_rows(monkeypatch):
    """What Int8Linear hands to moe_quantize_act, which reads M * K bf16 values from
    the address it gets: anything else is refused first."""
    import torch
    from quantized_moe_grouped_top_amd import runner
    calls = []
    monkeypatch.setattr(runner, "moe_quantize_act", lambda *a: calls.append(a))
    lin = runner.Int8Linear(4, 32, 16, device="cpu")
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    w, s = torch.zeros(16, 32, dtype=torch.int8), torch.zeros(16)
    for bad in (x.float(), x.half(), x[:3], x[:, :16], torch.zeros(8, 32, dtype=torch.bfloat16)[::2],
                torch.zeros(32, 4, dtype=torch.bfloat16).t(), x.view(-1), x.to("meta")):
        with pytest.raises(AssertionError):
            lin.quantize(bad)
        with pytest.raises(AssertionError):
            lin.forward(bad, w, s)
    assert not calls
    lin.quantize(x)
    lin.quantize(x.view(torch.int16))
    lin.quantize(x.view(2, 2, 32))
    assert len(calls) == 3


@needs_lib
@no_gpu
def test_layer_refuses_a_shared_expert_of_other_sizes(monkeypatch):
    """Before anything is enqueued: the layer would overwrite its results first."""
    import torch
    from quantized_moe_grouped_top_amd import runner
    calls = []
    for name in ("moe_align_block_size", "moe_quantize_act", "moe_grouped_gemm_int8w8a8", "moe_combine",
                 "moe_gemm_int8w8a8"):
        monkeypatch.setattr(runner, name, lambda *a, name=name: calls.append(name))
    moe = runner.RoutedMoE("int8dq", 4, 32, 16, 8, 2, device="cpu")
    x, logits = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 8)
    w, s = torch.zeros(8, 16, 32, dtype=torch.int8), torch.zeros(8, 16)
    for M, K, N, out in ((8, 32, 16, "bf16"), (4, 64, 16, "bf16"), (4, 32, 8, "bf16"), (4, 32, 16, "f32"),
                         (4, 32, 16, "f16")):
        lin = runner.Int8Linear(M, K, N, out=out, device="cpu")
        with pytest.raises(AssertionError):
            moe.forward(x, logits, w, s, shared=(lin, torch.zeros(N, K, dtype=torch.int8), torch.zeros(N)))
    assert not calls
    lin = runner.Int8Linear(4, 32, 16, device="cpu")
    moe.forward(x, logits, w, s, shared=(lin, w[0], s[0]))
    assert calls == ["moe_align_block_size", "moe_quantize_act", "moe_grouped_gemm_int8w8a8", "moe_combine",
                     "moe_quantize_act", "moe_gemm_int8w8a8"]


@needs_lib
@no_gpu
def test_router_aligns_into_whole_int32_buffers_only(monkeypatch):
    """The alignment writes max_padded slots and as many labels as blocks; what
    cannot hold them is refused first."""
    import torch
    from quantized_moe_grouped_top_amd import runner
    calls = []
    monkeypatch.setattr(runner, "moe_align_topk_ids", lambda *a: calls.append(a))
    r = runner.TopKRouter(40, 8, 2, device="cpu")
    n = qm.moe_align_max_padded(40, 8, 2, 16)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32)  # noqa: E731
    good = (i32(n), i32(n // 16), i32(1))
    for at, bad in ((0, i32(n - 1)), (0, i32(n).long()), (0, i32(2 * n)[::2]), (1, i32(n // 16 - 1)),
                    (1, i32(n // 16).short()), (1, i32(n // 16, 2)[:, 0]), (2, i32(0)), (2, torch.zeros(1))):
        buffers = list(good)
        buffers[at] = bad
        with pytest.raises(AssertionError):
            r.align(16, *buffers)
    with pytest.raises(qm.MoeError):
        r.align(24, *good)
    assert not calls
    r.align(16, *good)
    r.align(16, i32(n + 5), i32(n), i32(2))
    assert len(calls) == 2


@needs_lib
@no_gpu
@pytest.mark.parametrize("first,n_local,holds_all", [
    (0, None, True), (0, 8, True), (0, 4, False), (4, 4, False), (4, None, False), (6, 4, False),
    (0, 12, True), (-2, 10, True), (-2, 8, False)])
def test_rows_of_experts_elsewhere_are_cleared_for_every_window(monkeypatch, first, n_local, holds_all):
    """A window that misses an expert, however many it holds itself: the rows of y
    that no grouped GEMM writes must not reach the sum."""
    import torch
    from quantized_moe_grouped_top_amd import runner
    for name in ("moe_route_topk", "moe_align_topk_ids"):
        monkeypatch.setattr(runner, name, lambda *a: None)
    r = runner.TopKRouter(4, 8, 2, expert_first=first, n_local=n_local, device="cpu")
    moe = runner.RoutedMoE("int8dq", 4, 32, 16, r.n_local, 2, device="cpu", router=r)
    moe.y.fill_(7)
    moe.route(torch.zeros(4, 8))
    assert torch.all(moe.y == (7 if holds_all else 0))


@needs_lib
@no_gpu
def test_no_tokens_is_valid():
    assert _route(M=0, logits=None, topk_ids=None, topk_weights=None) == qm.MOE_OK
    assert _bwd(M=0, logits=None, d_logits=None) == qm.MOE_OK
    assert _int8(M=0, a_q=None, out=None) == qm.MOE_OK


@needs_lib
@no_gpu
def test_host_tensors_are_refused():
    import torch
    x = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(qm.MoeError) as ei:
        qm.moe_route_topk(x, 0, 8, None, 4, 8, 2, 0, 1, 1, 0, 1, 1.0, ids, w, stream=0)
    assert ei.value.code == INV


# ---- the oracle ------------------------------------------------------------------
def test_oracle_route_is_the_plain_router_without_extras():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 16)).astype(np.float32)
    x[3] = 0.25                                                  # all equal: lower experts first
    ids, w = L.route_general(x, None, 4)
    ids0, w0 = O.route_topk(x, 4)
    assert np.array_equal(ids, ids0)
    np.testing.assert_allclose(w, w0, rtol=1e-6)


@pytest.mark.parametrize("score", [L.SOFTMAX, L.SIGMOID])
@pytest.mark.parametrize("rule", [L.GROUP_MAX, L.GROUP_TOP2])
def test_oracle_route_groups_by_enumeration(score, rule):
    """Every choice of groups tried: the kept ones have the largest worths."""
    from itertools import combinations
    rng = np.random.default_rng(5)
    x, b = rng.standard_normal((30, 12)), 0.3 * rng.standard_normal(12)
    ids, w = L.route_general(x, b, 3, score, 4, 2, rule, True, 2.0)
    s = 1 / (1 + np.exp(-x)) if score == L.SIGMOID else np.exp(x) / np.exp(x).sum(1, keepdims=True)
    k = s + b
    for t in range(30):
        top = -np.sort(-k[t].reshape(4, 3), axis=1)
        worth = top[:, 0] if rule == L.GROUP_MAX else top[:, 0] + top[:, 1]
        best = max(combinations(range(4), 2), key=lambda c: worth[list(c)].sum())
        pool = [e for e in range(12) if e // 3 in best]
        want = sorted(pool, key=lambda e: -k[t, e])[:3]
        assert list(ids[t]) == want
        np.testing.assert_allclose(w[t], 2.0 * s[t, want] / s[t, want].sum(), rtol=1e-12)


@pytest.mark.parametrize("score", [L.SOFTMAX, L.SIGMOID])
def test_oracle_masked_experts_are_not_chosen(score):
    """A -inf logit takes its expert out whatever its bias: the choice of the
    router without these experts, which then have no group to lift either."""
    rng = np.random.default_rng(11)
    x, b = rng.standard_normal((20, 16)), 0.2 * rng.standard_normal(16)
    gone = np.array([1, 6, 8, 15])
    left = np.setdiff1d(np.arange(16), gone)
    x[:, 0] = -90.0                          # the same sigmoid score as -inf's in most formats
    x[:, gone], b[gone] = -np.inf, 0.9
    for n, keep, rule in ((1, 1, L.GROUP_MAX), (4, 2, L.GROUP_MAX), (4, 2, L.GROUP_TOP2)):
        ids, w = L.route_general(x, b, 4, score, n, keep, rule)
        want, w0 = L.route_general(x[:, left], b[left], 4, score, n, keep, rule)
        assert np.array_equal(ids, left[want])
        np.testing.assert_allclose(w, w0, rtol=1e-12)


def test_oracle_softmax_scores_of_a_token_with_a_nan():
    """The weights are NaN whether the NaN or +inf logit's expert is chosen or not."""
    x = np.zeros((3, 16))
    x[0, 10], x[1, 10] = np.nan, np.inf
    for bias in (None, np.zeros(16), 0.1 * np.arange(16.0)):
        for renorm in (True, False):
            ids, w = L.route_general(x, bias, 4, L.SOFTMAX, renormalize=renorm)
            assert np.isnan(w[:2]).all() and np.isfinite(w[2]).all()


@pytest.mark.parametrize("score", [L.SOFTMAX, L.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(7)
    x, g = rng.standard_normal((3, 10)), rng.standard_normal((3, 4))
    ids = np.argsort(-x, axis=1)[:, :4].astype(np.int32)

    def value(x):
        s = 1 / (1 + np.exp(-x)) if score == L.SIGMOID else np.exp(x) / np.exp(x).sum(1, keepdims=True)
        w = np.take_along_axis(s, ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return 1.5 * (w * g).sum()

    got = L.route_backward(g, ids, x, score, renorm, 1.5)
    h = 1e-5
    for t in range(3):
        for e in range(10):
            d = np.zeros_like(x)
            d[t, e] = h
            # central differences: h^2 f''' / 6 + eps / h, both below 1e-9 here
            assert abs((value(x + d) - value(x - d)) / (2 * h) - got[t, e]) < 1e-8


def test_oracle_gradient_of_the_smallest_sigmoid_scores():
    g = np.array([[1.0, -2.0, 0.5]])
    for v in (-700.0, -715.0, -740.0):
        got = L.route_backward(g, np.array([[2, 0, 5]]), np.full((1, 8), v), L.SIGMOID, True, 1.5)
        want = np.zeros((1, 8))
        want[0, [2, 0, 5]] = 0.5 * (g[0] - g[0].mean())
        np.testing.assert_allclose(got, want, rtol=1e-12)


def test_oracle_align_ids():
    rng = np.random.default_rng(1)
    ids = rng.integers(0, 8, (37, 2)).astype(np.int32)
    s, e, n, c = L.align_ids(ids, 8, 16)
    s0, e0, n0 = O.align_block_size(ids, 8, 16)
    assert np.array_equal(s, s0) and np.array_equal(e, e0) and n == int(np.ravel(n0)[0])
    assert np.array_equal(c, np.bincount(ids.ravel(), minlength=8))
    s, e, n, c = L.align_ids(ids, 4, 16, expert_first=2)          # experts 2..5 only
    assert c.sum() == np.isin(ids, [2, 3, 4, 5]).sum() and (s < 74).sum() == c.sum()
