"""The dense int8 product on the GPU against the float64 oracle (its integer
sums are exact there), and the layer that runs it beside the routed experts.

Tolerance.  The kernel's sum is exact; float(sum) is rounded once, then each of
the two scales, the bias and the addend round once more: 2^-24 of the
magnitude reached so far each, at most 5 * 2^-24 of the sum of the magnitudes;
then half a step of the output type."""

import zlib

import numpy as np
import pytest
import torch

import quantized_moe_grouped_top_amd as qm
from oracle import formats as F
from oracle import layer as L
from oracle import moe as O
from quantized_moe_grouped_top_amd import runner, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": (0, torch.float32), "bf16": (1, torch.bfloat16), "f16": (2, torch.float16)}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def _gen(*what):
    return torch.Generator().manual_seed(zlib.crc32(repr(what).encode()) & 0x7FFFFFFF)


def _codes(rows, K, ld, off, g):
    """int8 codes [rows, K], rows ld bytes apart, the first at byte `off` of its buffer."""
    flat = torch.randint(-128, 128, (rows * ld + off + 16,), generator=g, dtype=torch.int8).to(DEV)
    return flat[off:off + rows * ld].view(rows, ld)[:, :K]


def _rows_to_check(M, n=24):
    if M <= 2 * n:
        return np.arange(M)
    return np.unique(np.r_[0:n // 2, np.linspace(0, M - 1, n).astype(int), M - n // 2:M])


def check(M, K, N, out="bf16", bias=False, addend=False, pad=(0, 0, 0), off=(0, 0), ws=True,
          inplace=False, stream=None):
    print(f"\n[int8] M={M} K={K} N={N} {out} bias={bias} addend={addend} pad={pad} off={off} "
          f"ws={ws}", flush=True)
    g = _gen(M, K, N, out, pad, off)
    lda, ldw, ldo = K + pad[0], K + pad[1], N + pad[2]
    a, w = _codes(M, K, lda, off[0], g), _codes(N, K, ldw, off[1], g)
    sa = (torch.rand(M, generator=g) + 0.5).to(DEV) * (1.0 / 128)
    sw = (torch.rand(N, generator=g) + 0.5).to(DEV) * (1.0 / (128 * K ** 0.5))
    b = torch.randn(N, generator=g).to(DEV) if bias else None
    dt = DT[out][1]
    y = torch.full((M + 1, ldo), 5.0, dtype=dt, device=DEV)
    add = None
    if addend:
        add = torch.randn(M + 1, ldo, generator=g).to(dt).to(DEV)
        if inplace:
            y[:M, :N] = add[:M, :N]
    wb = qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N)
    scratch = torch.full((wb + 16,), 0x5A, dtype=torch.uint8, device=DEV) if ws else None
    qm.moe_gemm_int8w8a8(a, lda, sa, w, ldw, sw, b, y if inplace else add, M, K, N, DT[out][0], y,
                         ldo, scratch, stream=stream)
    torch.cuda.synchronize()
    assert torch.all(y[M] == 5.0) and torch.all(y[:M, N:] == 5.0)      # nothing but the outputs
    if ws:
        assert torch.all(scratch[wb:] == 0x5A)
    rows = _rows_to_check(M)
    cols = np.unique(np.r_[_rows_to_check(N, 300)]) if N > 600 else np.arange(N)
    ref, mag = L.gemm_int8(a.cpu().numpy()[rows], sa.cpu().numpy()[rows], w.cpu().numpy()[cols],
                           sw.cpu().numpy()[cols], None if b is None else b.cpu().numpy()[cols],
                           None if add is None else
                           add.double().cpu().numpy()[np.ix_(rows, cols)])
    got = y.double().cpu().numpy()[np.ix_(rows, cols)]
    tol = 5 * 2.0 ** -24 * mag
    tol = tol + torch.finfo(dt).eps / 2 * (np.abs(ref) + tol) + TINY[out]
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
    return a, sa, w, sw, y


SHAPES = [(1, 64, 16), (1, 4096, 4096), (1, 1, 1), (2, 17, 3), (3, 4096, 1024), (4, 128, 640),
          (5, 1000, 333), (8, 14336, 64), (15, 192, 2048), (16, 4096, 4096), (17, 512, 129),
          (31, 96, 257), (32, 2048, 1000), (33, 320, 64), (64, 4096, 2048), (65, 4096, 300),
          (100, 144, 1111), (127, 640, 512), (128, 4096, 1024), (129, 64, 255), (200, 1536, 777),
          (256, 256, 256), (257, 384, 513), (300, 4160, 1100), (511, 128, 520), (640, 1024, 640),
          (1000, 2048, 1500), (1030, 272, 2100), (2049, 512, 2304)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_int8_sizes(M, K, N):
    check(M, K, N)
    check(M, K, N, out="f32", bias=True, ws=False)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 512), (7, 1531, 401), (40, 768, 640), (130, 1531, 523),
                                   (300, 640, 770), (520, 4096, 1040)])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_int8_epilogue_and_strides(M, K, N, out):
    check(M, K, N, out, bias=True, addend=True)
    check(M, K, N, out, addend=True, inplace=True, pad=(16, 32, 8))
    check(M, K, N, out, bias=True, pad=((-K) % 16, (-K) % 16, 3))      # K inside aligned rows
    check(M, K, N, out, pad=(5, 1, 1), off=(3, 7))                     # nothing aligned
    check(M, K, N, out, pad=((-K) % 16, (-K) % 16 + 4, 0), off=(0, 0)) # one operand aligned
    check(M, K, N, out, pad=((-K) % 16, (-K) % 16, 0), off=(0, 8), ws=False)


@pytest.mark.parametrize("M", [1, 4, 16, 48, 64, 128, 192, 256, 384, 768])
@pytest.mark.parametrize("K,N", [(2048, 1024), (4096, 200), (144, 4096)])
def test_int8_rows(M, K, N):
    check(M, K, N)


@pytest.mark.parametrize("M,K,N", [(1, 14336, 256), (3, 12101, 124), (12, 8200, 300), (20, 6160, 96),
                                   (64, 14336, 1024), (33, 8192, 130), (100, 16384, 64)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_int8_shares_of_k(M, K, N, out):
    """Shapes whose contraction is shared out through the workspace."""
    assert qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N) > 0
    check(M, K, N, out, bias=True, addend=True)
    check(M, K, N, out, pad=(3, 5, 1), off=(1, 2))
    check(M, K, N, out, pad=((-K) % 16, (-K) % 16, 0), ws=False)


@pytest.mark.parametrize("M,K,N", [(384, 14336, 2050), (500, 16402, 1025), (385, 30007, 515), (512, 131071, 130)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_int8_shares_of_k_in_large_tiles(M, K, N, out):
    """128 x 128 tiles in shares, rows and columns that end inside one."""
    check(M, K, N, out, bias=True, addend=True, pad=((-K) % 16, (-K) % 16, 0))
    check(M, K, N, out, addend=True, inplace=True, pad=(3, 5, 1), off=(1, 2))
    check(M, K, N, out, pad=((-K) % 16, (-K) % 16, 0), ws=False)


@pytest.mark.parametrize("M,K,N", [(4352, 64, 4352), (4300, 80, 4400), (4352, 40, 4357), (4353, 200, 4352),
                                   (2500, 336, 9000)])
def test_int8_several_tiles_a_workgroup(M, K, N):
    check(M, K, N)
    check(M, K, N, "f32", bias=True, pad=((-K) % 16, (-K) % 16, 1))


@pytest.mark.parametrize("K", [16, 17, 31, 32, 48, 63, 65, 112, 127, 129, 143, 144, 240, 271, 1040])
def test_int8_ends_of_rows(K):
    """Every kernel's last, shorter step, in aligned rows and in rows at any byte."""
    for M, N in [(2, 40), (13, 90), (30, 130), (60, 200), (600, 1100), (1500, 1600)]:
        check(M, K, N, pad=((-K) % 16, (-K) % 16, 0))
        check(M, K, N, "f32", pad=(1, 1, 0), off=(1, 1))


@pytest.mark.parametrize("K", [1, 2, 7, 8, 15])
@pytest.mark.parametrize("M,N", [(1, 1), (63, 65), (64, 64), (130, 300), (1000, 70)])
def test_int8_rows_shorter_than_16(M, K, N):
    """The kernel of short rows: tiles that end inside rows and columns, rows at any
    byte, what lies behind the K bytes not read into the sums."""
    check(M, K, N)
    check(M, K, N, "f32", bias=True, addend=True, pad=(16 - K, 3, 1), off=(3, 1), ws=False)


def test_int8_two_streams():
    """Two calls at once, each with its own workspace, on two streams."""
    print("\n[int8] two streams", flush=True)
    M, K, N = 40, 14336, 512
    g = _gen("two")
    outs, refs, keep = [], [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        a, w = _codes(M, K, K, 0, g), _codes(N, K, K, 0, g)
        one = torch.ones(max(M, N), device=DEV)
        ws = torch.empty(qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N), dtype=torch.uint8, device=DEV)
        ref = torch.empty(M, N, device=DEV)
        qm.moe_gemm_int8w8a8(a, K, one, w, K, one, None, None, M, K, N, 0, ref, N, None)
        keep.append((a, w, one, ws))
        refs.append(ref)
        outs.append(torch.empty(M, N, device=DEV))
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            a, w, one, ws = keep[i]
            qm.moe_gemm_int8w8a8(a, K, one, w, K, one, None, None, M, K, N, 0, outs[i], N, ws,
                                 stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], refs[i])


def test_int8_kernels_in_a_graph():
    """The kernels of all sizes captured once and replayed on changing inputs."""
    print("\n[int8] graph", flush=True)
    g = _gen("graphs")
    work = []
    for M, K, N in [(1, 14336, 256), (64, 512, 1024), (300, 640, 2048), (1200, 256, 3000)]:
        a, w = _codes(M, K, K, 0, g), _codes(N, K, K, 0, g)
        sa, sw = torch.rand(M, generator=g).to(DEV), torch.rand(N, generator=g).to(DEV)
        ws = torch.empty(qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N) + 16, dtype=torch.uint8, device=DEV)
        work.append((M, K, N, a, w, sa, sw, ws, [torch.zeros(M, N, device=DEV) for _ in range(2)]))

    def step(k):
        for M, K, N, a, w, sa, sw, ws, y in work:
            qm.moe_gemm_int8w8a8(a, K, sa, w, K, sw, None, None, M, K, N, 0, y[k], N, ws)

    step(0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(1)
    for r in range(3):
        for M, K, N, a, *_ in work:
            a.copy_(torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8))
        step(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for M, K, N, *_, y in work:
            assert torch.equal(y[0], y[1]), (r, M, K, N)


def test_int8_extreme_codes():
    """All codes -128 at the largest K: the sum 128 * 128 * K is just below 2^31."""
    print("\n[int8] extreme", flush=True)
    K = qm.MOE_MAX_INT8_K
    for M in (1, 3, 20, 150):
        for ld in (K, K + 1):                                         # unaligned, aligned rows
            a = torch.full((M, ld), -128, dtype=torch.int8, device=DEV)
            w = torch.full((40, ld), -128, dtype=torch.int8, device=DEV)
            one = torch.ones(max(M, 40), device=DEV)
            y = torch.empty(M, 40, device=DEV)
            wb = qm.moe_gemm_int8w8a8_workspace_bytes(M, K, 40)
            ws = torch.empty(wb + 16, dtype=torch.uint8, device=DEV)
            qm.moe_gemm_int8w8a8(a, ld, one, w, ld, one, None, None, M, K, 40, 0, y, 40, ws)
            torch.cuda.synchronize()
            assert torch.all(y == float(np.float32(128 * 128 * K))), (M, ld)


def test_int8_is_exact_and_repeatable():
    """Unit scales: float32 outputs are the integers; with and without the
    workspace, and twice, the same bits."""
    print("\n[int8] exact", flush=True)
    for M, K, N in [(1, 4096, 768), (6, 4096, 256), (40, 4096, 512), (130, 2048, 256), (600, 1024, 512)]:
        g = _gen(M, K, N)
        a = torch.randint(-16, 17, (M, K), generator=g, dtype=torch.int8).to(DEV)
        w = torch.randint(-16, 17, (N, K), generator=g, dtype=torch.int8).to(DEV)
        one = torch.ones(max(M, N), device=DEV)
        wb = qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N)
        ws = torch.empty(wb + 16, dtype=torch.uint8, device=DEV)
        ref = a.cpu().double().numpy() @ w.cpu().double().numpy().T    # below 2^24: exact in float32
        for scratch in (ws, ws, None):
            y = torch.empty(M, N, device=DEV)
            qm.moe_gemm_int8w8a8(a, K, one, w, K, one, None, None, M, K, N, 0, y, N, scratch)
            torch.cuda.synchronize()
            assert np.array_equal(y.cpu().numpy().astype(np.float64), ref)


@pytest.mark.parametrize("M,K,N", [(5, 9, 70), (100, 15, 300), (1, 4096, 512), (1, 14336, 256),
                                   (40, 14336, 130), (64, 640, 1024), (300, 1024, 1100),
                                   (512, 14336, 1030), (1500, 272, 2100)])
def test_int8_epilogue_is_float32_in_its_order(M, K, N):
    """float(sum) * a_scale * w_scale + bias + addend, each step rounded to
    float32: the same bits from every kernel, with and without the workspace."""
    print(f"\n[int8] order M={M} K={K} N={N}", flush=True)
    g = _gen("order", M, K, N)
    a, w = _codes(M, K, K, 0, g), _codes(N, K, K, 0, g)
    sa = (torch.rand(M, generator=g) + 0.5).to(DEV) * (1.0 / 128)
    sw = (torch.rand(N, generator=g) + 0.5).to(DEV) * (1.0 / (128 * K ** 0.5))
    b, add = torch.randn(N, generator=g).to(DEV), torch.randn(M, N, generator=g).to(DEV)
    exact = a.cpu().double() @ w.cpu().double().t()               # integers below 2^53
    base = exact.float() * sa.cpu()[:, None] * sw.cpu()
    wb = qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N)
    ws = torch.empty(wb + 16, dtype=torch.uint8, device=DEV)
    for bias, addend in ((None, None), (b, None), (None, add), (b, add)):
        want = base if bias is None else base + b.cpu()
        want = want if addend is None else want + add.cpu()
        for scratch in (ws, None):
            y = torch.empty(M, N, device=DEV)
            qm.moe_gemm_int8w8a8(a, K, sa, w, K, sw, bias, addend, M, K, N, 0, y, N, scratch)
            torch.cuda.synchronize()
            assert torch.equal(y.cpu(), want), (bias is not None, addend is not None, scratch is not None)


def test_int8_large_output_offsets():
    """Output rows beyond 2^31 elements from the first: 64-bit offsets."""
    print("\n[int8] large output", flush=True)
    M, K, N, ldo = 520, 64, 256, (1 << 22) - 64
    g = _gen("large")
    a, w = _codes(M, K, K, 0, g), _codes(N, K, K, 0, g)
    one = torch.ones(M, device=DEV)
    y = torch.empty(M * ldo, dtype=torch.bfloat16, device=DEV)
    qm.moe_gemm_int8w8a8(a, K, one, w, K, one, None, None, M, K, N, 1, y, ldo, None)
    torch.cuda.synchronize()
    ref, mag = L.gemm_int8(a.cpu().numpy(), np.ones(M), w.cpu().numpy(), np.ones(N))
    got = torch.stack([y[m * ldo:m * ldo + N] for m in range(M)]).double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref) + 2.0 ** -22 * mag)


def test_on_another_stream_and_in_a_graph():
    """Route, align and int8 product on a side stream, captured and replayed
    with new inputs between the replays: each replay equals the eager run."""
    print("\n[layer] graph", flush=True)
    M, E, k, K, N = 96, 64, 4, 512, 384
    g = _gen("graph")
    x = torch.randn(M, E, generator=g).to(DEV)
    a, w = _codes(M, K, K, 0, g), _codes(N, K, K, 0, g)
    sa, sw = torch.rand(M, generator=g).to(DEV), torch.rand(N, generator=g).to(DEV)
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV)

    def buffers():
        n = qm.moe_align_max_padded(M, E, k, 16)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        return dict(ids=i32(M, k), w=torch.zeros(M, k, device=DEV), s=i32(n), e=i32(n // 16),
                    p=i32(1), c=i32(E), ws=i32(qm.moe_align_workspace_bytes(M, E, k) // 4),
                    dx=torch.zeros(M, E, device=DEV),
                    gw=torch.zeros(qm.moe_gemm_int8w8a8_workspace_bytes(M, K, N) + 16,
                                   dtype=torch.uint8, device=DEV),
                    y=torch.zeros(M, N, dtype=torch.bfloat16, device=DEV))

    def step(b):
        qm.moe_route_topk(x, 0, E, bias, M, E, k, 1, 8, 4, 1, 1, 2.5, b["ids"], b["w"])
        qm.moe_align_topk_ids(b["ids"], M, E, k, 16, 0, b["s"], b["e"], b["p"], b["c"], b["ws"])
        qm.moe_route_topk_backward(b["w"], b["ids"], x, 0, E, M, E, k, 1, 1, 2.5, b["dx"], E)
        qm.moe_gemm_int8w8a8(a, K, sa, w, K, sw, None, None, M, K, N, 1, b["y"], N, b["gw"])

    eager, cap = buffers(), buffers()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(cap)
    for r in range(4):
        x.copy_(torch.randn(M, E, generator=g))
        a.copy_(torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8))
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("ids", "w", "s", "e", "p", "c", "y", "dx"):
            assert torch.equal(eager[name], cap[name]), (r, name)


# ---- the layer -----------------------------------------------------------------------
@pytest.mark.parametrize("M,E,k,fmt,block_m", [(33, 16, 4, "int8dq", None), (300, 8, 2, "int8dq", 128),
                                               (64, 64, 6, "fp8", None)])
def test_layer_with_general_router_and_shared_expert(M, E, k, fmt, block_m):
    """RoutedMoE with the general router and an int8 shared expert: each stage
    against the oracle on the device's input of that stage."""
    print(f"\n[layer] M={M} E={E} k={k} {fmt}", flush=True)
    K, N = 256, 384
    g = _gen("layer", M, E)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(M, E, generator=g).to(torch.bfloat16).to(DEV)
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV)
    w = (torch.randn(E, N, K, generator=g) / K ** 0.5).to(DEV)
    wsh = (torch.randn(1, N, K, generator=g) / K ** 0.5).to(DEV)
    router = runner.TopKRouter(M, E, k, dtype="bf16", score="sigmoid", n_group=4, topk_group=3,
                               group_rule="top2", scale=2.5)
    shared = runner.Int8Linear(M, K, N)
    moe = runner.RoutedMoE(fmt, M, K, N, E, k, block_m=block_m, router=router)
    w_q, w_s = runner.quantize_weights(w, fmt)
    sh_q, sh_s = runner.quantize_weights(wsh, "int8")
    routed = moe.forward(x, logits, w_q, w_s, bias=bias).clone()
    out = moe.forward(x, logits, w_q, w_s, bias=bias, shared=(shared, sh_q[0], sh_s[0]))
    torch.cuda.synchronize()
    ids, wts = L.route_general(logits.float().cpu().numpy(), bias.cpu().numpy(), k, L.SIGMOID, 4, 3,
                               L.GROUP_TOP2, True, 2.5)
    assert np.array_equal(moe.topk_ids.cpu().numpy(), ids)
    np.testing.assert_allclose(moe.topk_weights.cpu().numpy(), wts, rtol=2.0 ** -23)
    s0, e0, p0, c0 = L.align_ids(ids, E, moe.block_m)
    assert np.array_equal(moe.sorted_token_ids.cpu().numpy(), s0)
    assert np.array_equal(moe.expert_ids.cpu().numpy(), e0)
    assert np.array_equal(router.expert_counts.cpu().numpy(), c0)
    # the routed experts on the device's quantized activations and weights
    aq, asc = moe.a_q.cpu().numpy(), moe.a_scale.cpu().numpy()
    if fmt == "int8dq":
        y = O.grouped_gemm_int8w8a8(aq, asc, w_q.cpu().numpy(), w_s.cpu().numpy(), ids,
                                    wts.astype(np.float32))
    else:
        y = O.grouped_gemm_fp8w8a8(aq, asc, w_q.cpu().numpy(), w_s.cpu().numpy(), ids,
                                   wts.astype(np.float32))
    got = F.bf16_decode(moe.y.cpu().numpy().view(np.uint16)).astype(np.float64)
    rms = np.sqrt(np.mean(y.astype(np.float64) ** 2))
    assert np.all(np.abs(got - y) <= 2e-2 * rms + 2.0 ** -8 * np.abs(y))
    # the shared expert on top of the routed sum
    base = F.bf16_decode(routed.cpu().numpy().view(np.uint16)).astype(np.float64)
    ref, mag = L.gemm_int8(shared.a_q.cpu().numpy(), shared.a_scale.cpu().numpy(),
                           sh_q[0].cpu().numpy(), sh_s[0].cpu().numpy(), None, base)
    fin = F.bf16_decode(out.cpu().numpy().view(np.uint16)).astype(np.float64)
    assert np.all(np.abs(fin - ref) <= 5 * 2.0 ** -24 * mag + 2.0 ** -8 * (np.abs(ref) + mag * 2.0 ** -21))
    # the router's gradient from the loss sum(out * r), through the per-slot results
    dw = torch.randn(M, k, generator=g).to(DEV)
    dx = router.backward(dw, logits)
    torch.cuda.synchronize()
    want = L.route_backward(dw.cpu().numpy(), ids, logits.float().cpu().numpy(), L.SIGMOID, True, 2.5)
    assert np.all(np.abs(dx.double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -40)


def test_layer_with_experts_on_two_devices():
    """The experts in two windows, as two devices hold them: every slot's result
    is the one of the layer that holds all, the other window leaves it zero, and
    the sums add up."""
    print("\n[layer] two windows", flush=True)
    M, E, k, K, N = 50, 16, 4, 256, 128
    g = _gen("windows")
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(M, E, generator=g).to(DEV)
    w = (torch.randn(E, N, K, generator=g) / 16).to(DEV)
    w_q, w_s = runner.quantize_weights(w, "int8dq")
    whole = runner.RoutedMoE("int8dq", M, K, N, E, k, router=runner.TopKRouter(M, E, k, score="sigmoid"))
    whole.forward(x, logits, w_q, w_s)
    total = torch.zeros(M * k, N, device=DEV)
    for first in (0, 8):
        router = runner.TopKRouter(M, E, k, score="sigmoid", expert_first=first, n_local=8)
        part = runner.RoutedMoE("int8dq", M, K, N, 8, k, router=router)
        part.forward(x, logits, w_q[first:first + 8], w_s[first:first + 8])
        torch.cuda.synchronize()
        here = ((router.topk_ids >= first) & (router.topk_ids < first + 8)).view(-1)
        assert torch.equal(part.y[here], whole.y[here]) and torch.all(part.y[~here] == 0)
        total += part.y.view(torch.bfloat16).float()
    assert torch.equal(total, whole.y.view(torch.bfloat16).float())


def test_quantized_linear_chain():
    """Int8Linear quantizes bf16 rows per token (the codes and scales of the
    oracle) and multiplies."""
    print("\n[layer] linear", flush=True)
    M, K, N = 45, 1024, 520
    x = synth.make_act_input(M, K, synth.seed_of("int8 linear"), std=1.0, device=DEV)
    w = (torch.randn(1, N, K, generator=_gen("lin")) / 32).to(DEV)
    q, s = runner.quantize_weights(w, "int8")
    lin = runner.Int8Linear(M, K, N, out="f32")
    y = lin.forward(x, q[0], s[0])
    torch.cuda.synchronize()
    aq, asc = O.quantize_act_int8_rows(x.view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(lin.a_q.cpu().numpy(), aq) and np.array_equal(lin.a_scale.cpu().numpy(), asc)
    ref, mag = L.gemm_int8(aq, asc, q[0].cpu().numpy(), s[0].cpu().numpy())
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= 4 * 2.0 ** -24 * mag)
