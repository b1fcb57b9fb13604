"""The block's norms, gate and residual on the GPU against the float64 reference.

Tolerance.  A row's mean of squares is a sum of N positive float32 terms, added in
a tree of at most 16 + 6 + 16 levels: 2^-18 of itself, and so are the factors;
each product and sum behind it rounds by 2^-24 of the magnitudes that go in, so 2^-18
of the sum of the magnitudes of an element's terms covers a row's values (2^-16 where
a row mean of products is among them, charged to the mean of their magnitudes).
Sums over tokens: (M / 512 + 140) additions of 2^-24 each, of the sum of magnitudes.
Then half a step of the output's type."""

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
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
GATES = {"none": 0, "channel": 1, "token": 2}
EPS = 1e-5
E1, E2 = 2.0 ** -18, 2.0 ** -16


def _rng(*what):
    return torch.Generator().manual_seed(zlib.crc32(repr(what).encode()) & 0x7FFFFFFF)


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, ref, err, dtype, what):
    got = _np(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    tol = err + HALF[dtype] * (np.abs(ref) + err) + TINY[dtype]
    worst = np.max(np.abs(got - ref) / tol) if ref.size else 0.0
    assert worst <= 1.0, (what, worst)


class Case:
    def __init__(self, M, N, k, dtype, r_dtype, post, gate, pre=True, block=True, residual=True,
                 alpha=0.8, beta=0.6, std=1.0):
        g = _rng(M, N, k, dtype, r_dtype, post, gate, pre, block, residual)
        t, rt = DT[dtype][1], DT[r_dtype][1]
        self.M, self.N, self.k, self.dtype, self.r_dtype = M, N, k, dtype, r_dtype
        self.kind, self.alpha, self.beta = GATES[gate], alpha, beta

        def rnd(*s, d=torch.float32, m=1.0, c=0.0):
            return (torch.randn(*s, generator=g) * m + c).to(d).to(DEV)

        self.y = rnd(M * k, N, d=t, m=std) if block else None
        self.x = rnd(M, N, d=rt, m=2.0) if residual else None
        self.w_post = rnd(N, m=0.2, c=0.5) if post else None
        self.w_pre = rnd(N, m=0.2, c=1.0) if pre else None
        self.gate = [None, rnd(N), rnd(M)][self.kind]
        self.d_r = rnd(M, N, d=rt)
        self.d_h = rnd(M, N, d=t) if pre else None

    def forward(self, stream=None, r=None, h=None):
        M, N = self.M, self.N
        r = torch.full((M + 1, N), 7.0, dtype=DT[self.r_dtype][1], device=DEV) if r is None else r
        if self.w_pre is not None and h is None:
            h = torch.full((M + 1, N), 7.0, dtype=DT[self.dtype][1], device=DEV)
        fo = torch.full((M + 1,), 7.0, device=DEV) if self.w_post is not None else None
        fr = torch.full((M + 1,), 7.0, device=DEV) if self.w_pre is not None else None
        qm.moe_norm_residual(self.y, DT[self.dtype][0], self.k, self.x, DT[self.r_dtype][0],
                             self.w_post, self.gate, self.kind, self.alpha, self.beta, self.w_pre,
                             EPS, M, N, r, h, fo, fr, stream=stream)
        return r, h, fo, fr

    def check_forward(self):
        M, N = self.M, self.N
        r, h, fo, fr = self.forward()
        rr, rh, rfo, rfr = B.norm_residual(_np(self.y), self.k, _np(self.x), _np(self.w_post),
                                           _np(self.gate), self.kind, self.alpha, self.beta,
                                           _np(self.w_pre), EPS, M, N)
        p = self._terms(rfo)[1]
        gate = 1.0
        if self.kind:
            gate = np.abs(_np(self.gate))
            gate = gate[None] if self.kind == 1 else gate[:, None]
        mag = self.beta * gate * p + (0 if self.x is None else self.alpha * np.abs(_np(self.x)))
        _close(r[:M], rr, E1 * mag, self.r_dtype, "r")
        assert bool((r[M:] == 7.0).all())
        if fo is not None:
            _close(fo[:M], rfo, E1 * rfo, "f32", "rstd_post")
            assert float(fo[M]) == 7.0
        if h is not None:
            # the mean of r^2 carries r's own error
            rel = E1 + 2 * E1 * (mag * np.abs(rr)).mean(1) / np.maximum((rr * rr).mean(1), 1e-30)
            _close(fr[:M], rfr, rel * rfr, "f32", "rstd_pre")
            w = np.abs(_np(self.w_pre))
            _close(h[:M], rh, w * rfr[:, None] * E1 * mag + np.abs(rh) * rel[:, None], self.dtype, "h")
            assert bool((h[M:] == 7.0).all())

    def _terms(self, f_post):
        """magnitudes of s (its slots') and p"""
        if self.y is None:
            z = np.zeros((self.M, self.N))
            return z, z
        s = np.abs(_np(self.y)).reshape(self.M, self.k, self.N).sum(1)
        if self.w_post is None:
            return s, s
        return s, np.abs(_np(self.w_post)) * s * f_post[:, None]

    def backward(self, d_r=True, stream=None):
        M, N = self.M, self.N
        r, _, fo, fr = self.forward()
        t, rt = DT[self.dtype][1], DT[self.r_dtype][1]
        self.r, self.fo, self.fr = r, fo, fr
        full = lambda *s, d=torch.float32: torch.full(s, 7.0, dtype=d, device=DEV)   # noqa: E731
        dx = full(M + 1, N, d=rt)
        dy = full(M + 1, N, d=t) if self.y is not None else None
        dwo = full(N + 1) if self.w_post is not None else None
        dwr = full(N + 1) if self.w_pre is not None else None
        dg = full([0, N, M][self.kind] + 1) if self.kind else None
        ws = torch.full((max(16, qm.moe_norm_backward_workspace_bytes(M, N)),), 0xFF,
                        dtype=torch.uint8, device=DEV)
        qm.moe_norm_residual_backward(self.d_r if d_r else None, self.d_h, self.y, DT[self.dtype][0],
                                      self.k, r, DT[self.r_dtype][0], self.w_post, self.gate,
                                      self.kind, self.alpha, self.beta, self.w_pre, fo, fr, M, N, dx,
                                      dy, dwo, dg, dwr, ws, stream=stream)
        return dx, dy, dwo, dg, dwr

    def check_backward(self, d_r=True):
        M, N = self.M, self.N
        dx, dy, dwo, dg, dwr = self.backward(d_r)
        cut = lambda v, n: None if v is None else _np(v)[:n]                         # noqa: E731
        fo, fr, r = cut(self.fo, M), cut(self.fr, M), cut(self.r, M)
        din = _np(self.d_r) if d_r else None
        ref = B.norm_residual_backward(din, _np(self.d_h), _np(self.y), self.k, r, _np(self.w_post),
                                       _np(self.gate), self.kind, self.alpha, self.beta,
                                       _np(self.w_pre), fo, fr, M, N)
        many = (M / 512 + 140) * 2.0 ** -24
        mdr = np.zeros((M, N)) if din is None else np.abs(din)
        if self.w_pre is not None:
            n, dh = np.abs(r) * fr[:, None], np.abs(_np(self.d_h))
            d = dh * np.abs(_np(self.w_pre))
            mdr = mdr + fr[:, None] * (d + n * (d * n).mean(1, keepdims=True))
            _close(dwr[:N], ref[4], (many + E1) * (dh * n).sum(0), "f32", "d_w_pre")
            assert float(dwr[N]) == 7.0
        _close(dx[:M], ref[0], E2 * self.alpha * mdr, self.r_dtype, "d_residual")
        assert bool((dx[M:] == 7.0).all())
        if self.y is None:
            return
        s, p = self._terms(fo)
        dq = self.beta * mdr
        dp = dq
        if self.kind:
            gate = np.abs(_np(self.gate))
            dp = dq * (gate[None] if self.kind == 1 else gate[:, None])
            if self.kind == 1:
                _close(dg[:N], ref[3], (many + E2) * (dq * p).sum(0), "f32", "d_gate")
            else:
                _close(dg[:M], ref[3], E2 * (dq * p).sum(1), "f32", "d_gate")
            assert float(dg[-1]) == 7.0
        err = E2 * dp
        if self.w_post is not None:
            m = s * fo[:, None]
            _close(dwo[:N], ref[2], (many + E2) * (dp * m).sum(0), "f32", "d_w_post")
            assert float(dwo[N]) == 7.0
            d = dp * np.abs(_np(self.w_post))
            err = E2 * fo[:, None] * (d + m * (d * m).mean(1, keepdims=True))
        _close(dy[:M], ref[1], err, self.dtype, "d_y")
        assert bool((dy[M:] == 7.0).all())


SIZES = [(1, 8, 1), (1, 4096, 2), (3, 16384, 8), (5, 520, 3), (64, 1032, 1), (130, 2056, 2),
         (517, 264, 1), (1100, 72, 1), (9, 8200, 1), (2, 512, 4)]


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                           ("f16", "f32")])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_norm_and_gradients(size, dtype, r_dtype, post, gate):
    M, N, k = size
    print(f"\n[norm] {size} {dtype} {r_dtype} post={post} gate={gate}", flush=True)
    c = Case(M, N, k, dtype, r_dtype, post, gate)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("kw", [
    dict(pre=False), dict(residual=False), dict(block=False, post=False, gate="none"),
    dict(pre=False, post=False, gate="channel"), dict(std=0.0), dict(std=1e4, post=False),
    dict(pre=False, residual=False, post=False, gate="none"),
], ids=str)
def test_parts_left_out(kw):
    args = dict(post=True, gate="token")
    args.update(kw)
    print(f"\n[norm] {args}", flush=True)
    c = Case(37, 264, 2, "bf16", "f32", **args)
    c.check_forward()
    c.check_backward()
    if c.w_pre is not None:
        c.check_backward(d_r=False)


def test_outputs_in_place():
    c = Case(33, 520, 1, "bf16", "bf16", True, "channel")
    r, h, _, _ = c.forward()
    dx, dy, dwo, dg, dwr = c.backward()
    x, y = c.x.clone(), c.y.clone()
    c.forward(r=c.x, h=c.y)
    assert torch.equal(c.x, r[:33]) and torch.equal(c.y, h[:33])
    c.x, c.y = x, y
    d = c.d_r.clone()
    ws = torch.empty(qm.moe_norm_backward_workspace_bytes(33, 520), dtype=torch.uint8, device=DEV)
    dy2 = torch.empty_like(dy)
    qm.moe_norm_residual_backward(d, c.d_h, c.y, 1, 1, c.r, 1, c.w_post, c.gate, 1, c.alpha, c.beta,
                                  c.w_pre, c.fo, c.fr, 33, 520, d, dy2, None, None, None, ws)
    assert torch.equal(d, dx[:33]) and torch.equal(dy2[:33], dy[:33])


def test_no_tokens():
    N = 64
    ws = torch.empty(16, dtype=torch.uint8, device=DEV)
    w = torch.ones(N, device=DEV)
    outs = [torch.full((N,), 7.0, device=DEV) for _ in range(3)]
    p = w.data_ptr()          # an array without elements has no address: any aligned one
    qm.moe_norm_residual(p, 1, 1, p, 1, w, w, 1, 1.0, 1.0, w, EPS, 0, N, p, p, None, None)
    qm.moe_norm_residual_backward(p, p, p, 1, 1, p, 1, w, w, 1, 1.0, 1.0, w, None, None, 0, N, None, p,
                                  outs[0], outs[1], outs[2], ws)
    for o in outs:
        assert not bool(o.any())


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_runner_of_no_tokens(gate):
    N, t = 72, torch.bfloat16
    norm = runner.BlockNorm(0, N, 2, gate=gate, train=True)
    y, x = torch.empty(0, N, dtype=t, device=DEV), torch.empty(0, N, dtype=t, device=DEV)
    w = torch.ones(N, device=DEV)
    g = {"none": None, "channel": w, "token": torch.empty(0, device=DEV)}[gate]
    for d in (norm.d_w_pre, norm.d_w_post, norm.d_gate):
        d.fill_(7.0)
    r, h = norm.forward(y, x, w, w, g)
    assert tuple(r.shape) == tuple(h.shape) == (0, N)
    _, _, d_pre, d_post, d_gate = norm.backward(x, x, y, w, w, g)
    for d in (d_pre, d_post, d_gate):
        assert d is None or not bool(d.any())


def test_a_row_of_infinities_stays_a_row():
    c = Case(20, 264, 1, "bf16", "f32", True, "none")
    r, h, _, _ = c.forward()
    c.y[7, 3] = float("inf")
    c.x[9, 0] = float("nan")
    r2, h2, _, _ = c.forward()
    rest = [t for t in range(20) if t not in (7, 9)]
    assert torch.equal(r2[rest], r[rest]) and torch.equal(h2[rest], h[rest])
    assert bool(torch.isnan(h2[9]).all())


def test_weight_gradients_repeat_and_many_rows():
    c = Case(3000, 264, 1, "bf16", "bf16", True, "channel")
    c.check_backward()
    first = c.backward()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.backward()))


def test_runner_block_norm():
    M, N = 40, 136
    c = Case(M, N, 2, "f16", "f32", True, "token")
    b = runner.BlockNorm(M, N, 2, "f16", "f32", "token", c.alpha, c.beta, EPS, train=True)
    r, h = b.forward(c.y, c.x, c.w_pre, c.w_post, c.gate)
    r0, h0, _, _ = c.forward()
    assert torch.equal(r, r0[:M]) and torch.equal(h, h0[:M])
    got = b.backward(c.d_r, c.d_h, c.y, c.w_pre, c.w_post, c.gate)
    dx, dy, dwo, dg, dwr = c.backward()
    for a, e, n in zip(got, (dx, dy, dwr, dwo, dg), (M, M, N, N, M)):
        assert torch.equal(a, e[:n])
    assert b.forward(c.y, c.x, None, None, c.gate)[1] is None
    with pytest.raises(AssertionError):
        b.forward(c.y, c.x, c.w_pre, c.w_post, None)
