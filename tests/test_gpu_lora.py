"""Low-rank adapters of many requests on the GPU against the float64 reference.

Tolerance.  v = A x: K products summed in float32 (K * 2^-23 of the magnitudes);
its two 16-bit parts leave out 2^-16 of v, and in fp16 2^-24 of the token's largest
value besides; B v: 2 R products summed in float32; the addend's sum and the scale
round once each; half a step of the output's type."""

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
U = 2.0 ** -23


def _rng(*what):
    return torch.Generator().manual_seed(zlib.crc32(repr(what).encode()) & 0x7FFFFFFF)


def _np(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, T, K, N, R, L, dtype, out, block_m, ids, ranks=True, scales=True, std=1.0):
        g = _rng(T, K, N, R, L, dtype, out, block_m)
        t = DT[dtype][1]
        self.T, self.K, self.N, self.R, self.L, self.dtype, self.out = T, K, N, R, L, dtype, out
        if ids == "random":
            self.ids = torch.randint(-1, L + 1, (T,), generator=g, dtype=torch.int32)
        elif ids == "runs":
            self.ids = (torch.arange(T) * L // T).int()
        else:
            self.ids = torch.full((T,), ids, dtype=torch.int32)
        self.x = torch.full((T, K + 8), float("nan"), dtype=t)
        self.x[:, :K] = (torch.randn(T, K, generator=g) * std).to(t)
        self.a = (torch.randn(L, R, K, generator=g) * K ** -0.5).to(t)
        self.b = (torch.randn(L, N, R, generator=g) * R ** -0.5).to(t)
        self.ranks = None
        if ranks:                                # what lies past a rank is never used
            self.ranks = torch.randint(0, R + 1, (L,), generator=g, dtype=torch.int32)
            for i, r in enumerate(self.ranks.tolist()):
                self.a[i, r:] = float("nan")
                self.b[i, :, r:] = float("nan")
        self.scales = torch.rand(L, generator=g) + 0.5 if scales else None
        self.add = torch.randn(T, N + 8, generator=g).to(DT[out][1])
        self.block_m = block_m
        for k in ("x", "a", "b", "ranks", "scales", "add"):
            v = getattr(self, k)
            setattr(self, k, None if v is None else v.to(DEV))
        self.ad = runner.LoraAdapters(T, K, R, L, dtype, block_m)
        self.ad.plan(self.ids.to(DEV))

    def reference(self, addend):
        xn, an, bn = _np(self.x)[:, :self.K], _np(self.a), _np(self.b)
        ids = self.ids.numpy()
        ranks = None if self.ranks is None else self.ranks.cpu().numpy()
        sc = None if self.scales is None else _np(self.scales)
        add = _np(self.add)[:, :self.N] if addend else None
        ref = B.lora(xn, an, bn, ids, ranks, sc, add)
        err = np.zeros_like(ref) if add is None else U * np.abs(add)
        for t, i in enumerate(ids):
            if 0 <= i < self.L:
                r = self.R if ranks is None else ranks[i]
                s = 1.0 if sc is None else sc[i]
                v = np.abs(an[i, :r] @ xn[t]) * s
                ev = self.K * U * (np.abs(an[i, :r]) @ np.abs(xn[t])) * s + 2.0 ** -16 * v
                ev += 2.0 ** -24 * (v.max() if r else 0.0)
                bm = np.abs(bn[i, :, :r])
                err[t] += bm @ ev + 2 * (self.R + 2) * U * (bm @ (v + ev))
        return ref, err

    def run(self, addend=True, inplace=False, stream=None):
        T, K, N, ad = self.T, self.K, self.N, self.ad
        out = self.add.clone() if inplace else torch.full((T, N + 8), 7.0, dtype=DT[self.out][1],
                                                          device=DEV)
        add = out if inplace else self.add if addend else None
        ws = torch.full((qm.moe_lora_workspace_bytes(T, K, self.R, self.L, self.block_m),), 0xFF,
                        dtype=torch.uint8, device=DEV)
        before = out.clone()
        qm.moe_lora_add(self.x, K + 8, self.a, self.b, self.ranks, self.scales, DT[self.dtype][0],
                        None if inplace else ad.adapter_ids, ad.sorted_token_ids, ad.expert_ids,
                        ad.num_tokens_post_padded, T, K, N, self.R, self.L, self.block_m, add,
                        DT[self.out][0], out, N + 8, ws, stream=stream)
        assert torch.equal(out[:, N:], before[:, N:])
        return out[:, :N]

    def check(self, addend=True, inplace=False):
        ref, err = self.reference(addend or inplace)
        got = _np(self.run(addend, inplace))
        assert np.isfinite(got).all()
        tol = err + HALF[self.out] * (np.abs(ref) + err) + TINY[self.out]
        worst = np.max(np.abs(got - ref) / tol)
        assert worst <= 1.0, worst


CASES = [
    (1, 8, 8, 8, 1, 16, 0), (1, 4096, 264, 16, 8, 16, 5), (1, 72, 72, 128, 3, 16, -1),
    (7, 264, 136, 24, 5, 16, "random"), (64, 1032, 520, 64, 100, 16, "random"),
    (64, 1032, 520, 64, 100, 16, 3), (100, 4104, 72, 8, 2, 32, "random"),
    (333, 200, 776, 40, 128, 64, "random"), (1000, 520, 264, 128, 3, 128, "runs"),
    (517, 64, 64, 16, 4, 256, "random"), (16, 128, 8, 8, 1, 16, 0), (17, 136, 16, 16, 1, 16, 0),
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                       ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_lora(case, dtype, out):
    T, K, N, R, L, block_m, ids = case
    print(f"\n[lora] {case} {dtype} {out}", flush=True)
    c = Case(T, K, N, R, L, dtype, out, block_m, ids)
    c.check()
    c.check(inplace=True)
    c.check(addend=False)


@pytest.mark.parametrize("T", [1, 40])
def test_lora_without_ranks_and_scales(T):
    Case(T, 520, 200, 32, 6, "bf16", "f32", 16, "random", False, False).check()


@pytest.mark.parametrize("std", [2.0 ** -18, 500.0])
def test_lora_of_small_and_large_inputs_in_fp16(std):
    """The inner vector leaves fp16's range or its normal numbers; the result does not."""
    Case(40, 520, 200, 32, 6, "f16", "f32", 16, "random", std=std).check()


def test_lora_infinite_input_stays_in_its_token():
    c = Case(20, 64, 72, 16, 2, "bf16", "f32", 16, "runs", False, False)
    good = c.run().clone()
    c.x[3, 5] = float("inf")
    c.x[11, 0] = float("nan")
    bad = c.run()
    rest = [t for t in range(20) if t not in (3, 11)]
    assert torch.equal(bad[rest], good[rest])
    assert not bool(torch.isfinite(bad[3]).any()) and bool(torch.isnan(bad[11]).all())


def test_labels_and_tokens_out_of_range_are_left_out():
    c = Case(20, 64, 72, 16, 2, "bf16", "bf16", 16, 1, False, False)
    c.ad.sorted_token_ids[0] = 1 << 30
    c.ad.sorted_token_ids[1] = -4
    c.ad.expert_ids[1] = 77
    out = c.run(inplace=True)
    first = c.ids.numel()
    keep = [0, 1] + list(range(16, first))            # named twice wrongly, in the block labelled 77
    assert torch.equal(out[keep], c.add[keep, :72])
    assert not torch.equal(out[2:16], c.add[2:16, :72])


def test_int8_linear_with_adapters():
    T, K, N, R, L = 33, 128, 200, 16, 3
    g = _rng("int8")
    lin = runner.Int8Linear(T, K, N)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(DEV)
    w_q, w_s = runner.quantize_weights((torch.randn(1, N, K, generator=g) * K ** -0.5).to(DEV), "int8")
    base = lin.forward(x, w_q[0], w_s[0]).clone()
    c = Case(T, K, N, R, L, "bf16", "bf16", 16, "random")
    got = lin.forward(x, w_q[0], w_s[0], lora=(c.ad, c.a, c.b, c.scales, c.ranks))
    c.x[:, :K] = x
    c.add[:, :N] = base
    assert torch.equal(got, c.run())
    with pytest.raises(AssertionError):
        lin.forward(x, w_q[0], w_s[0], lora=(c.ad, c.a, c.b[:, :64], c.scales, c.ranks))


def test_a_plan_for_more_features_serves_fewer():
    big = runner.LoraAdapters(9, 4096, 16, 4)
    ids = torch.arange(9, dtype=torch.int32, device=DEV) % 4
    big.plan(ids)
    c = Case(9, 264, 72, 16, 4, "bf16", "f32", 16, "random", False, False)
    small = runner.LoraAdapters(9, 264, 16, 4)
    small.plan(ids)
    x = c.x[:, :264]
    a = big.add(x, c.a, c.b, torch.empty(9, 72, device=DEV))
    b = small.add(x, c.a, c.b, torch.empty(9, 72, device=DEV))
    assert torch.equal(a, b)
    with pytest.raises(AssertionError):
        small.add(torch.zeros(9, 512, dtype=torch.bfloat16, device=DEV),
                  torch.zeros(4, 16, 512, dtype=torch.bfloat16, device=DEV), c.b, a)


def _split_case(dtype, out, below, T=24, R=16, N=128):
    """One adapter whose inner vector is known to the bit: v of rank r is an integer of
    24 bits times 2^(4 - below[r]) (a product of two full values and one of two small
    ones behind it), b has one power of two a column, scale is one: whatever is missing
    in the result was left out of v."""
    c = Case(T, 8, N, R, 1, dtype, out, 16, 0, ranks=False)
    bits = {"bf16": 8, "f16": 11}[dtype]
    g = _rng(dtype, out, tuple(below))
    lo, hi, small = 2 ** (bits - 1), 2 ** bits, {"bf16": 15, "f16": 1}[dtype]
    shift = 24 - 2 * bits                       # the second product stands that far behind
    big = torch.randint(lo, hi, (T,), generator=g).double()
    add = torch.randint(1, small + 1, (T,), generator=g).double()
    a0 = torch.randint(lo, hi, (R,), generator=g).double()
    a1 = 2.0 * torch.randint(0, 2 if dtype == "f16" else 8, (R,), generator=g).double() + 1.0
    unit = 2.0 ** (4 - torch.tensor([below[r % len(below)] for r in range(R)], dtype=torch.double))
    t = DT[dtype][1]
    x, a = torch.zeros(T, 8, dtype=torch.double), torch.zeros(R, 8, dtype=torch.double)
    x[:, 2], x[:, 5] = big, add
    a[:, 2], a[:, 5] = a0 * unit, a1 * unit * 2.0 ** -shift
    b = torch.zeros(N, R, dtype=torch.double)
    n = torch.arange(N)
    b[n, n % R] = 2.0 ** torch.randint(-2, 3, (N,), generator=g).double() * torch.where(n % 3 == 0, -1.0, 1.0)
    for v in (x, a, b):
        assert torch.equal(v, v.to(t).double())
    v = x @ a.t()
    assert torch.equal(v, v.float().double())
    c.x[:, :8], c.a[0], c.b[0] = x.to(t).to(DEV), a.to(t).to(DEV), b.to(t).to(DEV)
    scale = 2.0 ** {"bf16": -8, "f16": -14}[dtype]          # results in fp16's normal range
    c.scales[0] = scale
    return c, v.numpy(), (b * scale).numpy()


@pytest.mark.parametrize("below", [(0, 0, 1, 3), (0, 10, 6, 12), (0, 14, 16, 15), (0, 18, 20, 17)], ids=str)
@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("bf16", "f16")])
def test_what_is_left_out_of_the_inner_vector(dtype, out, below):
    """Two 16-bit parts leave out 2^-16 of a value of the inner vector (two steps of a
    half, bf16), three 2^-24 of it; in fp16 values reach down to 2^-39 of the token's
    largest besides: that is brought to 2^14 at least, where the smallest step of fp16
    is 2^-24 and half of it 2^-39 of 2^14.  No sum is in the way: every column has one
    product.  Then half a step of the output's type."""
    c, v, b = _split_case(dtype, out, below)
    left = (2.0 ** -24 if out == "f32" else 2.0 ** -16) * np.abs(v)
    if dtype == "f16":
        left += 2.0 ** -39 * np.abs(v).max(1, keepdims=True)
    ref, err = v @ b.T, left @ np.abs(b).T
    got = _np(c.run(addend=False))
    tol = err + HALF[out] * (np.abs(ref) + err)
    worst = np.max(np.abs(got - ref) / tol)
    assert worst <= 1.0, worst


def test_an_infinite_value_of_the_inner_vector_beside_large_ones_in_fp16():
    """inf b0 + 10^6 b1: an infinity of b0's sign, whatever sign b1 has."""
    c = Case(20, 8, 64, 16, 1, "f16", "f32", 16, 0, ranks=False, scales=False)
    c.x[:, :8] = 1000.0
    c.a[0].fill_(125.0)                          # v = 10^6, above fp16's largest value
    c.a[0, 3, 2] = float("inf")
    c.b[0] = torch.where(torch.rand(64, 16, generator=_rng("signs")) < 0.5, -1.0, 1.0).half().to(DEV)
    got = c.run(addend=False)
    want = c.b[0, :, 3].float() * float("inf")
    assert torch.equal(got, want.expand(20, 64))


@pytest.mark.parametrize("dtype,out,R", [("bf16", "bf16", 16), ("bf16", "f32", 64), ("f16", "f16", 128),
                                         ("f16", "f32", 24)])
def test_infinite_values_of_b(dtype, out, R):
    """v inf is an infinity of v's sign, also where v's later parts are 0 or of the other
    sign (v = 1, 1 - 2^-9 and such), NaN where v is 0; a NaN stays in its column."""
    T, N, rank = 40, 200, R - 3
    c = Case(T, 8, N, R, 2, dtype, out, 16, 1, ranks=False, scales=False)
    c.ranks = torch.tensor([R, rank], dtype=torch.int32, device=DEV)
    g = _rng("inf b", dtype, out)
    # x a: sums of a power of two and a small one either side of it; the last two tokens 0
    c.x[:, :8] = 0.0
    c.x[:T - 2, 0] = 1.0
    c.x[:T - 2, 1] = torch.tensor([0.0, 2.0 ** -9, -2.0 ** -9, 2.0 ** -13])[torch.arange(T - 2) % 4].to(DEV)
    sign = torch.where(torch.rand(R, generator=g) < 0.5, -1.0, 1.0)
    c.a[1, :, 0] = sign.to(DEV)
    c.a[1, :, 1] = 1.0
    c.b[1, 7, 3] = c.b[1, 150, rank - 1] = float("inf")
    c.b[1, 64, 0] = float("-inf")
    c.b[1, 65, 5], c.b[1, 65, 6] = sign[5] * float("inf"), sign[6] * float("inf")
    c.b[1, 199, 1] = float("nan")
    c.b[1, :, rank:] = float("inf")                       # past the rank: not used
    c.b[0] = float("inf")                                 # nobody's
    got = c.run(addend=True).double().cpu()
    n, m = torch.tensor([7, 150, 64, 65]), T - 2
    inf = float("inf")
    want = torch.stack([sign[3], sign[rank - 1], -sign[0], torch.ones(())]).double() * inf
    assert torch.equal(got[:m, n], want.expand(m, 4))
    assert bool(torch.isnan(got[m:, n]).all()) and bool(torch.isnan(got[:, 199]).all())
    rest = [i for i in range(N) if i not in (7, 150, 64, 65, 199)]
    c.b[1, [7, 150, 64, 65, 199]] = 0.0
    finite = c.run(addend=True).double().cpu()
    assert bool(torch.isfinite(finite).all()) and torch.equal(got[:, rest], finite[:, rest])


@pytest.mark.parametrize("T,block_m", [(255, 16), (256, 32), (1535, 32), (1536, 64)])
def test_blocks_that_the_runner_chooses(T, block_m):
    """Either side of each border: as with blocks given by hand, and right."""
    assert runner.LoraAdapters(T, 136, 24, 5).block_m == block_m
    Case(T, 136, 72, 24, 5, "bf16", "bf16", block_m, "random").check()
