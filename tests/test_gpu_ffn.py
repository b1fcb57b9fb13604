"""The experts' grouped 16-bit products on the GPU against the float64 reference.

Tolerance.  Products of 16-bit values are exact in float32; a sum of `depth` of
them in float32 is off by at most depth * 2^-24 of the sum of the magnitudes, twice
that where a matrix instruction cuts instead of rounding.  An activation's sigmoid
is off by (1 - s) (|z| + 4) 2^-22 of itself (the exponential's argument and its
value) and 2^-22 for the division; what this does to each output is carried
through by the product rule.  At the end half a step of the output's type."""

import zlib

import numpy as np
import pytest
import torch

import quantized_moe_grouped_top_amd as qm
from oracle import block as B
from quantized_moe_grouped_top_amd import runner

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": (0, torch.float32), "bf16": (1, torch.bfloat16), "f16": (2, torch.float16)}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
ACT = {"silu": 0, "gelu": 1}
U = 2.0 ** -23


def _rng(*what):
    return torch.Generator().manual_seed(zlib.crc32(repr(what).encode()) & 0x7FFFFFFF)


def _rows(shape, dtype, g, ld=None, std=1.0, live=None):
    """[rows, width] on the device, rows ld apart; NaN between the rows and in rows
    that no expert has."""
    rows, width = shape
    ld = ld or width
    t = torch.full((rows + 1, ld), float("nan"), dtype=DT[dtype][1])
    t[:rows, :width] = (torch.randn(rows, width, generator=g) * std).to(DT[dtype][1])
    if live is not None:
        t[:rows][~live] = float("nan")
    return t.to(DEV)[:rows, :width]


def _weights(E, N, K, dtype, g):
    return (torch.randn(E, N, K, generator=g) * K ** -0.5).to(DT[dtype][1]).to(DEV)


def _out(rows, width, dtype, ld=None):
    """Filled with a value that stays where nothing is written."""
    return torch.full((rows + 1, ld or width), 7.0, dtype=DT[dtype][1], device=DEV)


def _np(t):
    return np.nan_to_num(t.double().cpu().numpy(), nan=0.0)


def _offsets(splits, first=0):
    return torch.tensor(np.cumsum([first] + list(splits)), dtype=torch.int32, device=DEV)


def _live(splits, first, rows):
    v = torch.zeros(rows, dtype=torch.bool)
    v[first:first + sum(splits)] = True
    return v


def _close(got, ref, err, dtype, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    tol = err + HALF[dtype] * (np.abs(ref) + err) + TINY[dtype]
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.max(np.abs(got - ref) / tol)))


def _untouched(buf, written, what):
    """Every element outside `written` (rows, width) still holds the fill value."""
    rows, width = written
    keep = torch.ones(buf.shape, dtype=torch.bool, device=DEV)
    keep[rows, :width] = False
    assert bool((buf[keep] == 7.0).all()), f"{what}: written outside its rows"


# splits, rows before the first expert, rows behind the last, K, N
SHAPES = [
    ([1], 0, 0, 8, 8),
    ([1], 0, 0, 4096, 264),
    ([5, 0, 3], 0, 0, 40, 24),
    ([0, 0, 7], 2, 3, 64, 72),
    ([16, 17, 15, 1], 0, 1, 128, 136),
    ([33, 0, 64, 65], 1, 0, 264, 200),
    ([130, 0, 1, 257, 12], 0, 5, 328, 520),
    ([1] * 60 + [0] * 4, 0, 0, 96, 64),
    ([600, 300], 0, 0, 512, 776),
    ([1030, 0, 513, 255], 3, 2, 264, 1032),
    # 128 x 128 and 256 x 256 tiles in the one direction or the other, ends everywhere
    ([150, 0, 131, 257], 2, 1, 264, 2056),
    ([150, 131, 0, 257], 0, 3, 4104, 136),
    ([300, 0, 513, 259], 1, 0, 712, 8200),
    ([129, 385, 0, 558], 0, 2, 8200, 712),
    ([40, 0, 700, 1, 300], 0, 0, 2312, 2056),
    ([990], 7, 3, 136, 12200),
    ([900], 0, 100, 12200, 72),
]


def _setup(splits, before, behind, dtype):
    rows = before + sum(splits) + behind
    off = _offsets(splits, before)
    segs = B.segments(off.tolist(), rows)
    return rows, off, segs, _live(splits, before, rows)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_and_input_gradient(shape, dtype):
    splits, before, behind, K, N = shape
    print(f"\n[ffn] linear {shape} {dtype}", flush=True)
    g = _rng(shape, dtype)
    rows, off, segs, live = _setup(splits, before, behind, dtype)
    E = len(splits)
    w = _weights(E, N, K, dtype, g)
    x = _rows((rows, K), dtype, g, K + 8, live=live)
    y = _out(rows, N, dtype, N + 16)
    qm.moe_grouped_linear(x, K + 8, w, DT[dtype][0], off, rows, K, N, E, y, N + 16)
    xn, wn = _np(x), _np(w)
    ref = B.grouped_linear(xn, wn, segs, np.zeros((rows, N)))
    mag = B.grouped_linear(np.abs(xn), np.abs(wn), segs, np.zeros((rows, N)))
    m = live.numpy()
    _close(y[:rows, :N][live], ref[m], K * U * mag[m], dtype, "linear")
    rowmask = torch.cat([live, torch.zeros(1, dtype=torch.bool)]).to(DEV)
    _untouched(y, (rowmask, N), "linear")

    dy = _rows((rows, N), dtype, g, N + 8, live=live)
    dx = _out(rows, K, dtype, K + 8)
    qm.moe_grouped_linear_dgrad(dy, N + 8, w, DT[dtype][0], off, rows, K, N, E, dx, K + 8)
    dn = _np(dy)
    ref = B.grouped_dgrad(dn, wn, segs, np.zeros((rows, K)))
    mag = B.grouped_dgrad(np.abs(dn), np.abs(wn), segs, np.zeros((rows, K)))
    _close(dx[:rows, :K][live], ref[m], N * U * mag[m], dtype, "dgrad")
    _untouched(dx, (rowmask, K), "dgrad")


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_weight_gradient(shape, dtype, out):
    splits, before, behind, K, N = shape
    print(f"\n[ffn] wgrad {shape} {dtype} {out}", flush=True)
    g = _rng(shape, dtype, out)
    rows, off, segs, live = _setup(splits, before, behind, dtype)
    E = len(splits)
    x = _rows((rows, K), dtype, g, K + 8, live=live)
    dy = _rows((rows, N), dtype, g, N + 8, live=live)
    t = dtype if out == "same" else "f32"
    dw = torch.full((E * N * K + 64,), 7.0, dtype=DT[t][1], device=DEV)
    qm.moe_grouped_linear_wgrad(dy, N + 8, x, K + 8, DT[dtype][0], off, rows, K, N, E, DT[t][0], dw)
    xn, dn = _np(x), _np(dy)
    ref = B.grouped_wgrad(dn, xn, segs)
    mag = B.grouped_wgrad(np.abs(dn), np.abs(xn), segs)
    depth = np.array([hi - lo for lo, hi in segs])[:, None, None]
    _close(dw[:E * N * K].view(E, N, K), ref, depth * U * mag, t, "wgrad")
    assert bool((dw[E * N * K:] == 7.0).all())
    for e, (lo, hi) in enumerate(segs):
        if lo == hi:
            assert not bool(dw[e * N * K:(e + 1) * N * K].any()), "an expert without rows: 0"


def _act_error(gv, kind):
    """Errors of act(g) and act'(g) as the kernel evaluates them."""
    c = np.sqrt(2 / np.pi)
    z = gv if kind == 0 else 2 * c * (gv + 0.044715 * gv ** 3)
    dz = 1.0 if kind == 0 else 2 * c * (1 + 3 * 0.044715 * gv * gv)
    s = 1.0 / (1.0 + np.exp(-np.clip(z, -700, 700)))
    # of the sigmoid; below 2^-126 it may be 0 (the exponential's argument passes 87.3, its
    # value float32's range from 88.7 on), which is off by 2^-126 at most
    es = s * ((1 - s) * (np.abs(z) + 4) + 1) * 2.0 ** -22 + 2.0 ** -126
    a = np.abs(gv) * s
    ea = np.abs(gv) * es + a * 2.0 ** -23
    eda = es + np.abs(dz) * (ea * (1 - s) + a * (es + (1 - s) * 2.0 ** -21))
    return ea, eda


def _gated_up(splits, before, behind, K, H, dtype, act, keep=True, std=1.0):
    kind = ACT[act]
    g = _rng(splits, K, H, dtype, act)
    rows, off, segs, live = _setup(splits, before, behind, dtype)
    E = len(splits)
    w = _weights(E, 2 * H, K, dtype, g)
    x = _rows((rows, K), dtype, g, K + 16, std, live)
    gu = _out(rows, 2 * H, dtype) if keep else None
    h = _out(rows, H, dtype)
    qm.moe_gated_up(x, K + 16, w, DT[dtype][0], off, rows, K, H, E, kind, gu, h)
    xn, wn = _np(x), _np(w)
    rgu, rh = B.gated_up(xn, wn, segs, kind, np.zeros((rows, 2 * H)), np.zeros((rows, H)))
    err = K * U * B.grouped_linear(np.abs(xn), np.abs(wn), segs, np.zeros((rows, 2 * H)))
    m = live.numpy()
    rowmask = torch.cat([live, torch.zeros(1, dtype=torch.bool)]).to(DEV)
    if keep:
        _close(gu[:rows][live], rgu[m], err[m], dtype, "gu")
        _untouched(gu, (rowmask, 2 * H), "gu")
    eg, eu, u = err[:, :H], err[:, H:], np.abs(rgu[:, H:])
    ea = _act_error(rgu[:, :H], kind)[0] + 1.13 * eg          # |act'| <= 1.13
    e = ea * u + (np.abs(B.act(rgu[:, :H], kind)[0]) + ea) * eu + np.abs(rh) * U
    _close(h[:rows][live], rh[m], e[m], dtype, "h")
    _untouched(h, (rowmask, H), "h")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_up(shape, dtype, act):
    splits, before, behind, K, H = shape
    print(f"\n[ffn] up {shape} {dtype} {act}", flush=True)
    _gated_up(splits, before, behind, K, H, dtype, act)
    _gated_up(splits, before, behind, K, H, dtype, act, keep=False)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_up_of_large_inputs(act):
    """Gates of some hundred: the sigmoid is 0 or 1 and the exponential overflows."""
    print(f"\n[ffn] large {act}", flush=True)
    _gated_up([70, 30], 0, 0, 64, 72, "bf16", act, std=100.0)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_down_backward(shape, dtype, act, inplace):
    splits, before, behind, N, H = shape
    kind = ACT[act]
    print(f"\n[ffn] down backward {shape} {dtype} {act} {inplace}", flush=True)
    g = _rng(shape, dtype, act)
    rows, off, segs, live = _setup(splits, before, behind, dtype)
    E = len(splits)
    w = _weights(E, N, H, dtype, g)
    dy = _rows((rows, N), dtype, g, N + 8, live=live)
    gu = _rows((rows, 2 * H), dtype, g, std=2.0, live=live)
    rowmask = torch.cat([live, torch.zeros(1, dtype=torch.bool)]).to(DEV)
    dn, wn, gn = _np(dy), _np(w), _np(gu)
    if inplace:
        dgu, h = gu, None
    else:
        dgu, h = _out(rows, 2 * H, dtype), _out(rows, H, dtype)
    qm.moe_gated_down_backward(dy, N + 8, w, gu, DT[dtype][0], off, rows, N, H, E, kind, dgu, h)
    rd, rh = B.gated_down_backward(dn, wn, gn, segs, kind, np.zeros((rows, 2 * H)),
                                   np.zeros((rows, H)))
    dh = np.abs(B.grouped_dgrad(dn, wn, segs, np.zeros((rows, H))))
    edh = N * U * B.grouped_dgrad(np.abs(dn), np.abs(wn), segs, np.zeros((rows, H)))
    a, da = (np.abs(v) for v in B.act(gn[:, :H], kind))
    ea, eda = _act_error(gn[:, :H], kind)
    u = np.abs(gn[:, H:])
    e = np.concatenate([edh * u * (da + eda) + dh * u * eda, edh * (a + ea) + dh * ea], axis=1)
    m = live.numpy()
    _close(dgu[:rows][live], rd[m], (e + np.abs(rd) * U)[m], dtype, "dgu")
    if inplace:
        assert bool(torch.isnan(dgu[:rows][~live]).all()), "rows of no expert stay"
    else:
        _close(h[:rows][live], rh[m], (ea * u + np.abs(rh) * U)[m], dtype, "h")
        _untouched(dgu, (rowmask, 2 * H), "dgu")
        _untouched(h, (rowmask, H), "h")


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [([700, 0, 900], 1, 2, 1800, 6152), ([40, 0, 300, 1], 0, 1, 2056, 5000)],
                         ids=["many rows", "many tiles"])
def test_weight_gradient_in_the_large_tiles(shape, dtype, out):
    """256 x 256 tiles: more than 512 rows an expert, and more than 640 tiles."""
    test_weight_gradient(shape, dtype, out)


def test_one_expert_without_offsets_and_no_rows():
    g = _rng("dense")
    K, N, rows = 72, 80, 37
    w, x = _weights(1, N, K, "bf16", g), _rows((rows, K), "bf16", g)
    y, z = _out(rows, N, "bf16"), _out(rows, N, "bf16")
    off = _offsets([rows])
    qm.moe_grouped_linear(x, K, w, 1, None, rows, K, N, 1, y, N)
    qm.moe_grouped_linear(x, K, w, 1, off, rows, K, N, 1, z, N)
    assert torch.equal(y, z) and not bool((y[:rows] == 7.0).all())
    qm.moe_grouped_linear(None, K, w, 1, None, 0, K, N, 1, None, N)
    dw = torch.full((1, N, K), 7.0, dtype=torch.bfloat16, device=DEV)
    qm.moe_grouped_linear_wgrad(None, N, None, K, 1, None, 0, K, N, 1, 1, dw)
    assert not bool(dw.any())


def test_offsets_outside_the_rows_are_taken_to_their_ends():
    g = _rng("ends")
    rows, K, N, E = 40, 64, 72, 4
    off = torch.tensor([-5, 12, 12, 30, 1 << 30], dtype=torch.int32, device=DEV)
    segs = B.segments(off.tolist(), rows)
    assert segs == [(0, 12), (12, 12), (12, 30), (30, 40)]
    w, x = _weights(E, N, K, "bf16", g), _rows((rows, K), "bf16", g)
    y = _out(rows, N, "bf16")
    qm.moe_grouped_linear(x, K, w, 1, off, rows, K, N, E, y, N)
    xn, wn = _np(x), _np(w)
    ref = B.grouped_linear(xn, wn, segs, np.zeros((rows, N)))
    mag = B.grouped_linear(np.abs(xn), np.abs(wn), segs, np.zeros((rows, N)))
    _close(y[:rows], ref, K * U * mag, "bf16", "linear")
    _untouched(y, (slice(0, rows), N), "linear")


def test_rows_past_32_bit_offsets():
    """An array of 5.2 * 10^9 elements: rows 16384 elements apart."""
    K, N, ld, rows = 64, 16, 16384, 320000
    print("\n[ffn] 64-bit offsets", flush=True)
    g = _rng("wide")
    buf = torch.empty(rows, ld, dtype=torch.bfloat16, device=DEV)
    x = buf[:, :K]
    tail = (torch.randn(300, K, generator=g)).to(torch.bfloat16).to(DEV)
    x.zero_()
    x[-300:] = tail
    w = _weights(2, N, K, "bf16", g)
    off = torch.tensor([0, rows - 200, rows], dtype=torch.int32, device=DEV)
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    qm.moe_grouped_linear(x, ld, w, 1, off, rows, K, N, 2, y, N)
    tn, wn = _np(tail), _np(w)
    ref = np.concatenate([tn[:100] @ wn[0].T, tn[100:] @ wn[1].T])
    mag = np.concatenate([np.abs(tn[:100]) @ np.abs(wn[0]).T, np.abs(tn[100:]) @ np.abs(wn[1]).T])
    _close(y[-300:], ref, K * U * mag, "bf16", "far rows")
    assert not bool(y[:-300].any())
    dw = torch.empty(2, N, K, dtype=torch.float32, device=DEV)
    dy = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    d = torch.randn(300, N, generator=g).to(torch.bfloat16).to(DEV)
    dy[-300:] = d
    qm.moe_grouped_linear_wgrad(dy, N, x, ld, 1, off, rows, K, N, 2, 0, dw)
    dn = _np(d)
    ref = np.stack([dn[:100].T @ tn[:100], dn[100:].T @ tn[100:]])
    mag = np.stack([np.abs(dn[:100]).T @ np.abs(tn[:100]), np.abs(dn[100:]).T @ np.abs(tn[100:])])
    _close(dw, ref, 300 * U * mag, "f32", "far rows' gradient")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_runner_feed_forward_and_its_gradients(dtype):
    """GatedFFN's two passes against the reference fed with the stored 16-bit
    intermediate values, so that each step is measured on its own error."""
    splits, K, H = [40, 0, 129, 70], 136, 200
    rows, E = sum(splits), len(splits)
    g = _rng("runner", dtype)
    off = _offsets(splits)
    segs = B.segments(off.tolist(), rows)
    ffn = runner.GatedFFN(rows, K, H, E, dtype, "gelu", train=True, dw="f32")
    x, dy = _rows((rows, K), dtype, g), _rows((rows, K), dtype, g)
    w_up, w_down = _weights(E, 2 * H, K, dtype, g), _weights(E, K, H, dtype, g)
    y = ffn.forward(x, w_up, w_down, off)
    hn, wd = _np(ffn.h), _np(w_down)
    ref = B.grouped_linear(hn, wd, segs, np.zeros((rows, K)))
    mag = B.grouped_linear(np.abs(hn), np.abs(wd), segs, np.zeros((rows, K)))
    _close(y, ref, H * U * mag, dtype, "y")
    dx, dw_up, dw_down = ffn.backward(dy, x, w_up, w_down, off)
    dn, xn, dyn, wu = _np(ffn.dgu), _np(x), _np(dy), _np(w_up)
    ref = B.grouped_dgrad(dn, wu, segs, np.zeros((rows, K)))
    mag = B.grouped_dgrad(np.abs(dn), np.abs(wu), segs, np.zeros((rows, K)))
    _close(dx, ref, 2 * H * U * mag, dtype, "dx")
    for got, a, b, name in ((dw_up, dn, xn, "dw_up"), (dw_down, dyn, hn, "dw_down")):
        _close(got, B.grouped_wgrad(a, b, segs),
               129 * U * B.grouped_wgrad(np.abs(a), np.abs(b), segs), "f32", name)
    # the chain as a whole against float64 from the inputs alone: three 16-bit roundings
    gu, h = B.gated_up(xn, wu, segs, 1, np.zeros((rows, 2 * H)), np.zeros((rows, H)))
    dgu, _ = B.gated_down_backward(dyn, wd, gu, segs, 1, np.zeros((rows, 2 * H)), np.zeros((rows, H)))
    whole = B.grouped_dgrad(dgu, wu, segs, np.zeros((rows, K)))
    rms = np.sqrt((whole ** 2).mean())
    assert np.sqrt(((dx.double().cpu().numpy() - whole) ** 2).mean()) < 4 * HALF[dtype] * rms


def test_results_repeat():
    g = _rng("repeat")
    splits, K, H = [300, 40, 0, 900], 264, 520
    rows, E = sum(splits), 4
    ffn = runner.GatedFFN(rows, K, H, E, train=True)
    off = _offsets(splits)
    x, dy = _rows((rows, K), "bf16", g), _rows((rows, K), "bf16", g)
    w_up, w_down = _weights(E, 2 * H, K, "bf16", g), _weights(E, K, H, "bf16", g)
    first = None
    for _ in range(3):
        out = [ffn.forward(x, w_up, w_down, off), *ffn.backward(dy, x, w_up, w_down, off)]
        out = [t.clone() for t in out]
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradient_at_infinite_gates(dtype, act):
    """A gate that left its type's range on the way forward: act and act' have their
    limits there (0 and 0; an infinity and 1); a NaN stays one."""
    rows, N, H = 70, 72, 136
    g = _rng("infinite gates", dtype, act)
    w = _weights(1, N, H, dtype, g)
    dy, gu = _rows((rows, N), dtype, g), _rows((rows, 2 * H), dtype, g)
    inf = float("inf")
    gu[:, 3], gu[:, 60], gu[:, 135] = -inf, inf, float("nan")
    u = _np(gu)[:, H:]
    dgu, h = _out(rows, 2 * H, dtype), _out(rows, H, dtype)
    qm.moe_gated_down_backward(dy, N, w, gu, DT[dtype][0], None, rows, N, H, 1, ACT[act], dgu, h)
    dg, du, h = dgu[:rows, :H], dgu[:rows, H:], h[:rows]
    assert not bool(dg[:, 3].any()) and not bool(du[:, 3].any()) and not bool(h[:, 3].any())
    dn, wn = _np(dy), _np(w)[0]
    dh, mag = dn @ wn, np.abs(dn) @ np.abs(wn)
    _close(dg[:, 60], dh[:, 60] * u[:, 60], N * U * (mag[:, 60] * np.abs(u[:, 60])), dtype, "dg")
    assert np.array_equal(du[:, 60].double().cpu().numpy(), np.sign(dh[:, 60]) * inf)
    assert np.array_equal(h[:, 60].double().cpu().numpy(), np.sign(u[:, 60]) * inf)
    for t in (dg, du, h):
        assert bool(torch.isnan(t[:, 135]).all())
        rest = [i for i in range(H) if i not in (3, 60, 135)]
        assert bool(torch.isfinite(t[:, rest]).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_past_a_gate_below_fp16(act):
    """One token's gate of -80000 is -inf in fp16's gu and its h is 0: it adds nothing,
    neither to its own gradient nor to the weights' (these in float32: the token's other
    gates, 266 * 400 in float64, are above fp16's 65504)."""
    rows, K, H = 40, 72, 40
    g = _rng("below", act)
    ffn = runner.GatedFFN(rows, K, H, 1, "f16", act, train=True, dw="f32")
    x, dy = _rows((rows, K), "f16", g), _rows((rows, K), "f16", g)
    w_up, w_down = _weights(1, 2 * H, K, "f16", g), _weights(1, K, H, "f16", g)
    x[:, 0], x[7, 0] = 0.0, 400.0
    w_up[0, 9, 0] = -200.0
    y = ffn.forward(x, w_up, w_down).clone()
    assert float(ffn.gu[7, 9]) == -float("inf") and float(ffn.h[7, 9]) == 0.0
    grads = [t.clone() for t in ffn.backward(dy, x, w_up, w_down)]
    assert all(bool(torch.isfinite(t).all()) for t in [y] + grads)
    assert float(ffn.dgu[7, 9]) == 0.0 and float(ffn.dgu[7, H + 9]) == 0.0
