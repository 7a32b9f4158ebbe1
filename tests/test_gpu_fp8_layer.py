"""The layer on 8-bit codes against its definitions in 64 bits, at the sizes,
masks and values where it can go wrong.

Bounds.  A code is within half a step of its value: 2^-4 of it, or half the
smallest subnormal, 2^-10, times the scale.  expf is within 2^-23 relative
(1 ulp), so sigmoid in fp32 is within 4 * 2^-24 of the exact one (exp, sum,
quotient) and SiLU(g) u within 7 * 2^-24; its gradient's longest path, dh u s (1
+ g (1 - s)), adds five roundings and the error of 1 - s and is held to 2^-20
(|dh u s| (1 + |g|)).  A sum of n exact products on the tensor cores is taken to
be within n 2^-23 sum |terms|, which also covers truncation instead of rounding;
sums over blocks in fp32 add one rounding per block and two for the scales.
Every output lies between guard values."""

import math

import numpy as np
import pytest
import torch

from nvfp4_mixture_experts_counting_gb300 import ftmoe

from test_gpu_train_ops import (BF16, DEV, EPS, FP16, FP32, NAMES, TINY, UNIT, Guarded, built, gen, randn,  # noqa: F401
                                tables, within)

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
CODE, CODE_TINY = 2.0 ** -4, 2.0 ** -10  # half a step: relative, and of a subnormal
TYPES = pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=lambda d: NAMES[d])


def blocks(n):
    return -(-n // 128)


def ratio(a, b):
    """a / b rounded once: torch multiplies by the reciprocal where one of them is a number."""
    full = lambda v, like: v if torch.is_tensor(v) else torch.full_like(like, v)
    return full(a, b) / full(b, a)


def quantized(x):
    """(codes, scales) by the header's formula, in fp32."""
    rows, n = x.shape
    x = torch.nn.functional.pad(x.float(), (0, blocks(n) * 128 - n)).view(rows, blocks(n), 128)
    top = x.abs().amax(2, keepdim=True)
    scale = torch.where(top < 1e-30, 0.0, ratio(top, 448))
    mul = torch.where(top < 1e-30, 0.0, ratio(448, top))
    return (x * mul).to(E4M3).view(rows, -1)[:, :n].contiguous(), scale[:, :, 0].t().contiguous()


def value(codes, scales):
    """What codes [rows, n] and scales [ceil(n/128), rows] stand for, in 64 bits."""
    n = codes.shape[1]
    return codes.double() * scales.double().t().repeat_interleave(128, 1)[:, :n]


def bank(g, E, N, K, std=0.05):
    w = torch.nn.functional.pad(randn(g, E, N, K, std=std), (0, blocks(K) * 128 - K, 0, blocks(N) * 128 - N))
    w = w.view(E, blocks(N), 128, blocks(K), 128)
    top = w.abs().amax((2, 4), keepdim=True)
    codes = (w * ratio(448, top)).to(E4M3).view(E, blocks(N) * 128, -1)[:, :N, :K].contiguous()
    return codes, ratio(top, 448)[:, :, 0, :, 0].contiguous()


def bank_value(codes, scales):
    E, N, K = codes.shape
    return codes.double() * scales.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]


def rows_of(g, M, width):
    """Codes and scales of rows of different sizes, one of them zeros."""
    x = randn(g, M, width) * torch.exp(randn(g, M, 1))
    if M > 2:
        x[1] = 0
    return quantized(x)


def same_codes(got, want):
    """Equal as bytes, but for the sign of NaN."""
    a, b = got.float(), want.float()
    assert bool(((a == b) | (a.isnan() & b.isnan())).all())


# ----------------------------------------------------------------- quantisers

@TYPES
@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (3, 144), (17, 640), (5, 2000), (64, 2560), (2, 8208)])
def test_quantize_rows(T, K, dtype):
    g, new = gen(1), Guarded()
    x = (randn(g, T, K) * torch.exp(2 * randn(g, T, 1))).to(dtype)
    x[0, :16] = 0
    codes, scales = new((T, K), E4M3), new((blocks(K), T), FP32)
    ftmoe.ftmoe_fp8_quantize(x, T, K, None, 1, codes, scales)
    want, scale = quantized(x)
    same_codes(codes, want)
    assert torch.equal(scales, scale)
    new.check()
    bound = CODE * x.double().abs() + CODE_TINY * scale.double().t().repeat_interleave(128, 1)[:, :K]
    within(value(codes, scales), x.double(), bound * (1 + 1e-6))


def test_quantize_special_values():
    """Zeros, the threshold, tiny, huge, infinite and NaN blocks."""
    x = torch.zeros(8, 256, device=DEV)
    x[1, 3], x[2, 3], x[3, 3] = 9.9e-31, 1.01e-30, -3e38
    x[4, 3], x[5, 3], x[6, 3] = math.inf, math.nan, -math.inf
    x[4:7, 128:] = 1.0
    x[7] = torch.linspace(-1, 1, 256, device=DEV)
    new = Guarded()
    codes, scales = new((8, 256), E4M3), new((2, 8), FP32)
    ftmoe.ftmoe_fp8_quantize(x, 8, 256, None, 1, codes, scales)
    want, scale = quantized(x)
    for r in (0, 1, 2, 3, 7):
        assert torch.equal(codes[r].view(torch.uint8) & 127, want[r].view(torch.uint8) & 127)
        assert torch.equal(scales[:, r], scale[:, r])
    assert scales[0, 0] == 0 and scales[0, 1] == 0 and scales[0, 2] > 0
    v = value(codes, scales)
    for r in (4, 5, 6):
        assert bool(v[r, 3].isnan()) and not bool(scales[0, r].isfinite())  # the block is spoiled
        assert bool(((v[r, 128:] - 1).abs() <= EPS).all())  # the other one is not; its scale is rounded
    new.check()


@TYPES
@pytest.mark.parametrize("T,k,E,K,drop", [(1, 1, 2, 16, 0.0), (16, 8, 64, 640, 0.0), (65, 6, 60, 2000, 0.3),
                                          (7, 32, 40, 144, 0.5)])
def test_quantize_into_expert_rows(T, k, E, K, drop, dtype):
    g, new = gen(2), Guarded()
    x = randn(g, T, K, dtype=dtype)
    idx = torch.argsort(torch.rand(T, E, generator=g, device=DEV), 1)[:, :k].int()
    idx[torch.rand(T, k, generator=g, device=DEV) < drop] = -1
    _, _, inv = tables(idx, E)
    inv = torch.as_tensor(inv, dtype=torch.int32, device=DEV)
    P = T * k
    codes, scales = new((P, K), torch.uint8, 9), new((blocks(K), P), FP32, 5.0)
    ftmoe.ftmoe_fp8_quantize(x, T, K, inv, k, codes, scales)
    want, scale = quantized(x)
    kept = torch.nonzero(inv >= 0)[:, 0]
    assert torch.equal(codes[inv[kept].long()], want.view(torch.uint8)[kept // k])
    assert torch.equal(scales[:, inv[kept].long()], scale[:, kept // k])
    left = torch.ones(P, dtype=torch.bool, device=DEV)
    left[inv[kept].long()] = False
    assert bool((codes[left] == 9).all()) and bool((scales[:, left] == 5.0).all())
    new.check()


def test_quantize_bad_places_and_counts():
    g, new = gen(3), Guarded()
    x = randn(g, 4, 128, dtype=BF16)
    inv = torch.tensor([0, 8, -2, 3, -1, 1, 2, 1 << 30], dtype=torch.int32, device=DEV)
    codes, scales = new((8, 128), torch.uint8, 9), new((1, 8), FP32, 5.0)
    ftmoe.ftmoe_fp8_quantize(x, 4, 128, inv, 2, codes, scales)
    assert ftmoe.ftmoe_ops_status() == -10
    want, scale = quantized(x)
    for at, t in ((0, 0), (3, 1), (1, 2), (2, 3)):
        assert torch.equal(codes[at], want.view(torch.uint8)[t]) and scales[0, at] == scale[0, t]
    assert bool((codes[4:] == 9).all())
    for n, rows, status in ((0, 0, 0), (3, 3, 0), (4, 4, 0), (5, 4, -10), (-1, 0, -10)):
        codes.fill_(9)
        ftmoe.ftmoe_fp8_quantize(x, 4, 128, None, 1, codes, scales,
                                 used=torch.tensor([n], dtype=torch.int32, device=DEV))
        assert ftmoe.ftmoe_ops_status() == status
        assert torch.equal(codes[:rows], want.view(torch.uint8)[:rows]) and bool((codes[rows:] == 9).all())
    new.check()


@TYPES
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (2, 130, 144), (3, 256, 640), (2, 999, 400)])
def test_quantize_weights(E, N, K, dtype):
    g, new = gen(4), Guarded()
    w = (randn(g, E, N, K) * torch.exp(randn(g, E, N, 1))).to(dtype)
    w[0, :128, :16] = 0
    codes, scales = new((E, N, K), E4M3), new((E, blocks(N), blocks(K)), FP32)
    ftmoe.ftmoe_fp8_quantize_weights(w, E, N, K, codes, scales)
    p = torch.nn.functional.pad(w.float(), (0, blocks(K) * 128 - K, 0, blocks(N) * 128 - N))
    p = p.view(E, blocks(N), 128, blocks(K), 128)
    top = p.abs().amax((2, 4), keepdim=True)
    want = torch.where(top < 1e-30, 0.0, p * ratio(448, top)).to(E4M3).view(E, blocks(N) * 128, -1)[:, :N, :K]
    same_codes(codes, want)
    assert torch.equal(scales, torch.where(top < 1e-30, 0.0, ratio(top, 448))[:, :, 0, :, 0])
    new.check()


# ----------------------------------------------------------------- SwiGLU

def silu_up(gu):
    g, u = gu.double().chunk(2, 1)
    return g * torch.sigmoid(g) * u


def silu_up_grad(dh, gu):
    g, u = gu.double().chunk(2, 1)
    d, s = dh.double(), torch.sigmoid(g)
    exact = torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], 1)
    return exact, torch.cat([(d * u * s).abs() * (1 + g.abs()), (d * g * s).abs()], 1) * 2.0 ** -20


@TYPES
@pytest.mark.parametrize("rows,I", [(1, 1), (1, 8), (33, 7), (65, 129), (16, 640), (257, 1001)])
def test_swiglu(rows, I, dtype):
    g, new = gen(5), Guarded()
    gu = randn(g, rows, 2 * I, dtype=dtype, std=3.0)
    gu[0, 0], gu[0, I] = -200.0, 2.0
    out = new((rows, I), dtype)
    ftmoe.ftmoe_swiglu(gu, rows, I, out)
    exact = silu_up(gu)
    within(out, exact, UNIT[dtype] * exact.abs() + TINY[dtype] + 8 * EPS * exact.abs())
    dh, dgu = randn(g, rows, I, dtype=dtype), new((rows, 2 * I), dtype)
    ftmoe.ftmoe_swiglu_backward(dh, gu, rows, I, dgu)
    exact, bound = silu_up_grad(dh, gu)
    within(dgu, exact, UNIT[dtype] * exact.abs() + TINY[dtype] + 2 * bound)
    here = gu.clone()
    ftmoe.ftmoe_swiglu_backward(dh, here, rows, I, here)  # in its input's place
    assert torch.equal(here, dgu)
    new.check()


@TYPES
@pytest.mark.parametrize("rows,I", [(1, 128), (33, 640), (130, 384)])
def test_swiglu_to_codes(rows, I, dtype):
    g, new = gen(6), Guarded()
    gu, dh = randn(g, rows, 2 * I, dtype=dtype, std=2.0), randn(g, rows, I, dtype=dtype)
    gu[rows - 1, I:I + 128] = 0  # a block of zeros
    codes, scales = new((rows, I), E4M3), new((I // 128, rows), FP32)
    ftmoe.ftmoe_swiglu(gu, rows, I, codes, scales)
    exact = silu_up(gu)
    top = exact.abs().view(rows, -1, 128).amax(2).t() / 448
    within(scales, top, 12 * EPS * top)
    wide = top.t().repeat_interleave(128, 1)
    within(value(codes, scales), exact, (CODE * exact.abs() + CODE_TINY * wide) * (1 + 2.0 ** -16) + 12 * EPS * exact.abs())
    assert float(scales[0, rows - 1]) == 0.0
    codes, scales = new((rows, 2 * I), E4M3), new((2 * I // 128, rows), FP32)
    ftmoe.ftmoe_swiglu_backward(dh, gu, rows, I, codes, scales)
    exact, bound = silu_up_grad(dh, gu)
    wide = (exact.abs().view(rows, -1, 128).amax(2) / 448).repeat_interleave(128, 1)
    spread = bound.view(rows, -1, 128).amax(2).repeat_interleave(128, 1) * 2  # of the value, and of the scale's
    within(value(codes, scales), exact, (CODE * exact.abs() + CODE_TINY * wide) * (1 + 2.0 ** -16) + 2 * spread)
    new.check()


def test_swiglu_leaves_rows_behind_the_last():
    g, new = gen(7), Guarded()
    gu = randn(g, 40, 256, dtype=BF16)
    gu[10:] = math.nan
    used = torch.tensor([10], dtype=torch.int32, device=DEV)
    out, codes, scales = new((40, 128), BF16, 3.0), new((40, 128), torch.uint8, 9), new((1, 40), FP32, 5.0)
    ftmoe.ftmoe_swiglu(gu, 40, 128, out, used=used)
    ftmoe.ftmoe_swiglu(gu, 40, 128, codes, scales, used=used)
    assert bool((out[10:] == 3.0).all()) and bool((codes[10:] == 9).all()) and bool((scales[:, 10:] == 5.0).all())
    assert bool(out[:10].isfinite().all()) and bool(scales[:, :10].isfinite().all())
    new.check()


# ----------------------------------------------------------------- the product

def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)


def product(a, a_scale, w, w_scale, counts, transpose):
    """Exact product and its error bound in fp32, row by row of each expert; rows of no expert are 0."""
    x, wv = value(a, a_scale), bank_value(w, w_scale)
    M, (E, N, K) = a.shape[0], w.shape
    y = torch.zeros(M, K if transpose else N, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(y)
    at = 0
    for e, n in enumerate(counts):
        r = slice(at, at + n)
        m = wv[e] if transpose else wv[e].t()
        y[r], mag[r] = x[r] @ m, x[r].abs() @ m.abs()
        at += n
    return y, (128 + blocks(N if transpose else K) + 4) * 2.0 ** -23 * mag


def run_product(a, a_scale, w, w_scale, counts, dtype, transpose=False, out=None, new=None):
    M, (E, N, K) = a.shape[0], w.shape
    new = new or Guarded()
    out = new((M, K if transpose else N), dtype, 7.0) if out is None else out
    ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, offsets_of(counts), M, E, N, K, out, transpose=transpose)
    new.check()
    return out


COUNTS = [
    # M, counts of each expert
    (1, [1]), (1, [0, 1, 0]), (5, [2, 0, 3]), (40, [17, 0, 1, 22]), (64, [0, 0, 64]), (300, [129, 1, 127, 43]),
    (1000, [700, 0, 300]), (37, [10, 7, 3]),  # the last leaves rows of no expert
    (63, [0] * 20 + [37, 0, 0, 23] + [0] * 9), (90, [1, 0, 2] * 30), (700, [0] * 300 + [1] * 500 + [200]),
]
SHAPES = [(16, 16), (128, 128), (144, 272), (256, 640), (333, 400), (640, 2000), (1280, 2560), (96, 4112)]


@pytest.mark.parametrize("M,counts", COUNTS, ids=lambda v: str(v) if isinstance(v, int) else "")
@pytest.mark.parametrize("N,K", SHAPES)
def test_product(N, K, M, counts):
    g = gen(10 + N + K + M)
    a, a_scale = rows_of(g, M, K)
    w, w_scale = bank(g, len(counts), N, K)
    y, bound = product(a, a_scale, w, w_scale, counts, False)
    out = run_product(a, a_scale, w, w_scale, counts, FP32)
    n = sum(counts)
    within(out[:n], y[:n], bound[:n] + TINY[FP32])
    assert bool((out[n:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("M,counts", [(40, [17, 0, 1, 22]), (300, [129, 1, 127, 43])])
def test_product_rounds_once(M, counts, dtype):
    g = gen(20)
    a, a_scale = rows_of(g, M, 400)
    w, w_scale = bank(g, len(counts), 333, 400, std=0.02)
    y, bound = product(a, a_scale, w, w_scale, counts, False)
    out = run_product(a, a_scale, w, w_scale, counts, dtype)
    within(out, y, UNIT[dtype] * y.abs() + TINY[dtype] + bound * (1 + UNIT[dtype]))


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("N", [8, 16, 24, 48, 80])
def test_product_of_many_narrow_tiles(N, dtype):
    """Hundreds of short tiles a CTA: none goes out from shared memory that the next one writes."""
    g = gen(25 + N)
    M, K = 2_000_000, 16
    a, a_scale = rows_of(g, M, K)
    w, w_scale = bank(g, 1, N, K)
    y, bound = product(a, a_scale, w, w_scale, [M], False)
    for _ in range(3):
        out = run_product(a, a_scale, w, w_scale, [M], dtype)
        unit = UNIT.get(dtype, 0.0)
        within(out, y, unit * y.abs() + TINY[dtype] + bound * (1 + unit))


@pytest.mark.parametrize("M,counts", COUNTS, ids=lambda v: str(v) if isinstance(v, int) else "")
@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (144, 272), (640, 400), (1280, 2560)])
def test_product_with_columns(N, K, M, counts):
    """The gradient of the input."""
    g = gen(30 + N + K + M)
    a, a_scale = rows_of(g, M, N)
    w, w_scale = bank(g, len(counts), N, K)
    y, bound = product(a, a_scale, w, w_scale, counts, True)
    n = sum(counts)
    for dtype in (FP32, BF16):
        out = run_product(a, a_scale, w, w_scale, counts, dtype, transpose=True)
        within(out[:n], y[:n], bound[:n] * (1 + UNIT[dtype]) + UNIT[dtype] * y[:n].abs() + TINY[dtype])
        assert bool((out[n:] == 7.0).all())


@pytest.mark.parametrize("M,counts", COUNTS, ids=lambda v: str(v) if isinstance(v, int) else "")
@pytest.mark.parametrize("I,K", [(128, 16), (128, 272), (640, 2560), (384, 400)])
def test_product_with_swiglu(I, K, M, counts):
    g, new = gen(40 + I + K + M), Guarded()
    E = len(counts)
    a, a_scale = rows_of(g, M, K)
    w, w_scale = bank(g, E, 2 * I, K, std=0.1)
    y, bound = product(a, a_scale, w, w_scale, counts, False)
    codes, scales = new((M, I), E4M3), new((I // 128, M), FP32, 5.0)
    codes.view(torch.uint8).fill_(9)
    ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, offsets_of(counts), M, E, 2 * I, K, codes, scales, swiglu=True)
    new.check()
    n = sum(counts)
    assert bool((codes[n:].view(torch.uint8) == 9).all()) and bool((scales[:, n:] == 5.0).all())
    gate, up = y[:n].chunk(2, 1)
    dg, du = bound[:n].chunk(2, 1)
    h = silu_up(y[:n])
    # |d SiLU| <= 1.1; the rest as for SwiGLU itself
    err = 1.1 * dg * (up.abs() + du) + (gate * torch.sigmoid(gate)).abs() * du + 8 * EPS * h.abs()
    worst = err.view(n, -1, 128).amax(2)
    top = h.abs().view(n, -1, 128).amax(2)
    within(scales[:, :n].t(), top / 448, (worst + 2 * EPS * top) / 448 + 1e-30)
    wide = (top / 448).repeat_interleave(128, 1)
    spread = worst.repeat_interleave(128, 1)
    within(value(codes[:n], scales[:, :n]), h,
           (CODE * h.abs() + CODE_TINY * wide) * (1 + 2.0 ** -16) + 2 * err + 2 * spread + 1e-30)


def test_product_without_offsets():
    g = gen(50)
    a, a_scale = rows_of(g, 70, 272)
    w, w_scale = bank(g, 1, 144, 272)
    y, bound = product(a, a_scale, w, w_scale, [70], False)
    new = Guarded()
    out = new((70, 144), FP32)
    ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, None, 70, 1, 144, 272, out)
    within(out, y, bound + TINY[FP32])
    new.check()


def test_product_with_bad_offsets():
    """An expert whose rows fall or leave the matrix is left out and marked; the others are computed."""
    g = gen(51)
    a, a_scale = rows_of(g, 20, 128)
    w, w_scale = bank(g, 4, 128, 128)
    good = run_product(a, a_scale, w, w_scale, [5, 5, 5, 5], FP32)
    out = torch.full((20, 128), 7.0, device=DEV)
    for bad in ([0, 5, 10, 9, 20], [0, 5, 10, 21, 20], [0, 5, 10, -4, 20], [0, 5, 10, 1 << 30, -(1 << 30)]):
        out.fill_(7.0)
        ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, torch.tensor(bad, dtype=torch.int32, device=DEV), 20, 4, 128,
                               128, out)
        assert ftmoe.ftmoe_ops_status() == -10
        assert torch.equal(out[:10], good[:10])


def test_product_keeps_rows_apart():
    """NaN and infinite scales in one row, or in rows of no expert, reach no other row."""
    g = gen(52)
    counts = [3, 30, 0, 4]
    a, a_scale = rows_of(g, 50, 400)
    w, w_scale = bank(g, 4, 160, 400)
    good = run_product(a, a_scale, w, w_scale, counts, FP32)
    bad, bad_scale = a.clone(), a_scale.clone()
    bad.view(torch.uint8)[37:] = 0x7F  # NaN
    bad_scale[:, 37:] = math.inf
    bad.view(torch.uint8)[5, 7] = 0x7F
    bad_scale[1, 20] = math.inf
    out = run_product(bad, bad_scale, w, w_scale, counts, FP32)
    rows = [r for r in range(37) if r not in (5, 20)]
    assert torch.equal(out[rows], good[rows])
    assert bool(out[5].isnan().all()) and not bool(out[20].isfinite().any())


def test_product_repeats_bit_for_bit():
    g = gen(53)
    counts = [129, 1, 127, 43]
    a, a_scale = rows_of(g, 300, 2000)
    w, w_scale = bank(g, 4, 640, 2000)
    first = run_product(a, a_scale, w, w_scale, counts, FP32)
    for _ in range(3):
        assert torch.equal(run_product(a, a_scale, w, w_scale, counts, FP32), first)


# ----------------------------------------------------------------- routing

def route(logits, k, score="softmax", norm=True, scale=1.0, bias=None, groups=(1, 1, 1)):
    T, new = logits.shape[0], Guarded()
    idx, w = new((T, k), torch.int32), new((T, k), FP32)
    ftmoe.ftmoe_route_topk(ftmoe.route_args(logits, idx, w, score=score, norm_topk_prob=norm, scale=scale, bias=bias,
                                            n_groups=groups[0], top_groups=groups[1], group_best=groups[2]))
    new.check()
    return idx, w


def routed(logits, k, score, norm, scale, bias, groups):
    """The definition in numpy, in 64 bits; the least distance between values that decide, relative to them."""
    z = logits.double().cpu().numpy()
    T, E = z.shape
    G, top, best = groups
    b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
    idx, w, near = np.full((T, k), -1), np.zeros((T, k)), math.inf

    def least(v):
        """Of falling values; equal ones are ties, not neighbours."""
        v = v[np.isfinite(v)]
        gaps = (v[:-1] - v[1:]) / np.maximum(np.maximum(abs(v[:-1]), abs(v[1:])), 1e-300)
        return min([math.inf] + [x for x in gaps if x > 0])

    for t in range(T):
        on = np.isfinite(z[t]) & np.isfinite(b)
        zt = np.where(on, z[t], 0.0)
        if score == "sigmoid":
            s = np.exp(-np.logaddexp(0, -zt))
        else:
            usable = np.isfinite(z[t])
            s = np.exp(zt - z[t][usable].max()) / np.exp(z[t][usable] - z[t][usable].max()).sum() if usable.any() else zt
        rank = np.where(on, (zt if bias is None and (G == 1 or best == 1) else s + np.where(on, b, 0.0)), -np.inf)
        if G > 1:
            m = -np.sort(-rank.reshape(G, -1), 1)[:, :best]
            score_g = np.where(np.isfinite(m), m, 0).sum(1)
            score_g[~np.isfinite(m[:, 0])] = -np.inf
            order = np.argsort(-score_g, kind="stable")
            near = min(near, least(score_g[order][top - 1:top + 1]))
            keep = np.zeros(G, bool)
            keep[order[:top]] = True
            rank = np.where(np.repeat(keep, E // G), rank, -np.inf)
        order = np.argsort(-rank, kind="stable")
        near = min(near, least(rank[order][:k + 1]))
        n = min(k, int(np.isfinite(rank).sum()))
        idx[t, :n] = order[:n]
        chosen = order[:n]
        if n:
            if norm:  # ratios survive where scores underflow
                logs = -np.logaddexp(0, -zt[chosen]) if score == "sigmoid" else zt[chosen]
                p = np.exp(logs - logs.max())
                w[t, :n] = scale * p / p.sum()
            else:
                w[t, :n] = scale * s[chosen]
    return idx, w, near


def check_route(logits, k, score="softmax", norm=True, scale=1.0, bias=None, groups=(1, 1, 1), span=12.0):
    idx, w = route(logits, k, score, norm, scale, bias, groups)
    want, ww, near = routed(logits, k, score, norm, scale, bias, groups)
    assert near > 1e-13  # else 64 bits would not decide either
    assert np.array_equal(idx.cpu().numpy(), want)
    # exp (2 eps), its argument's rounding (span eps), sums and quotient: relative to the weight
    within(w, ww, (24 + 2 * span) * EPS * np.abs(ww) + 1e-37)
    return idx, w


ROUTES = [
    # T, E, k, groups (number, chosen, best)
    (1, 1, 1, (1, 1, 1)), (3, 2, 1, (1, 1, 1)), (17, 31, 5, (1, 1, 1)), (9, 33, 32, (1, 1, 1)), (64, 60, 6, (3, 2, 2)),
    (130, 256, 8, (8, 4, 2)), (33, 256, 8, (1, 1, 1)), (40, 100, 4, (10, 3, 1)), (16, 1024, 16, (32, 5, 2)),
    (5, 1000, 8, (1, 1, 1)), (12, 64, 8, (32, 4, 1)), (50, 28, 3, (7, 2, 2)), (11, 32, 4, (32, 4, 2)),
    (8, 512, 32, (2, 1, 2)),
]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups", ROUTES)
def test_route(T, E, k, groups, score, norm, biased):
    g = gen(60 + T + E)
    bias = randn(g, E, std=0.1) if biased else None
    check_route(randn(g, T, E, std=1.5), k, score, norm, 2.5, bias, groups)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_16_bit_logits_tie_often(score, dtype):
    g = gen(61)
    logits = randn(g, 200, 256, dtype=dtype)
    check_route(logits, 8, score)
    check_route(logits, 8, score, groups=(8, 4, 1))
    check_route(logits, 8, score, bias=torch.zeros(256, device=DEV), groups=(8, 4, 2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_values_closer_than_fp32(score):
    """Scores plus biases that fp32 cannot tell apart are ranked as in exact arithmetic."""
    g = gen(62)
    E, T = 64, 400
    logits = randn(g, T, E, std=1.0)
    for t in range(T):  # pairs one fp32 step apart, in either order
        i, j = (t * 7) % E, (t * 11 + 5) % E
        if i != j:
            logits[t, i] = 3.0 + 0.001 * t
            logits[t, j] = torch.nextafter(logits[t, i].cpu(), torch.tensor(9.0 if t % 2 else -9.0)).to(DEV)
    bias = torch.full((E,), 0.625, device=DEV)
    check_route(logits, 4, score, bias=bias)
    check_route(logits, 4, score, bias=bias, groups=(8, 4, 2))


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_closer_than_fp32(score, best):
    """Groups whose worth differs by one fp32 step of one logit, or not at all, and tokens of which all values do."""
    g = gen(66)
    T, E, G = 200, 96, 8
    logits = randn(g, T, E)
    z = logits.view(T, G, E // G)
    for t in range(T):
        z[t, (3 * t + 1) % G] = z[t, t % G]  # the same values, in another order
        z[t, (3 * t + 1) % G] = z[t, (3 * t + 1) % G].flip(0)
        if t % 3:
            at = int(z[t, t % G].argmax())
            z[t, t % G, at] = torch.nextafter(z[t, t % G, at].cpu(), torch.tensor(9.0 if t % 2 else -9.0)).to(DEV)
    bias = torch.full((E,), 0.375, device=DEV)
    check_route(logits, 5, score, bias=bias, groups=(G, 4, best))
    check_route(logits, 5, score, bias=bias, groups=(G, 1, best))
    steps = torch.randint(0, 4, (40, E), generator=g, device=DEV).int()
    near = (torch.full((40, E), 1.25, device=DEV).view(torch.int32) + steps).view(FP32)  # up to three steps apart
    check_route(near, 5, score, bias=bias, groups=(G, 4, best))
    check_route(near, 5, score, bias=bias)
    check_route(near, 32, score, bias=bias)
    check_route(near, 5, score)


def test_route_masked_and_bad_logits():
    inf, nan = math.inf, math.nan
    z = torch.full((6, 8), -inf, device=DEV)
    z[1, 5] = 2.0
    z[2, [1, 3, 6]] = torch.tensor([1.0, -1.0, 1.0], device=DEV)
    z[3] = torch.arange(8.0, device=DEV)
    z[5, 0], z[5, 7] = -300.0, -310.0
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(8, device=DEV)):
            for groups in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
                check_route(z, 4, score, bias=bias, groups=groups, span=320.0)
                assert ftmoe.ftmoe_ops_status() == 0
    # the type's lowest value is a value, not a mask
    low = torch.full((2, 8), torch.finfo(FP32).min, device=DEV)
    low[1, 2] = 0.0
    idx, w = route(low, 3)
    assert idx.tolist() == [[0, 1, 2], [2, 0, 1]] and w[1].tolist() == [1.0, 0.0, 0.0]
    within(w[0], torch.full((3,), 1 / 3, dtype=torch.float64), 4 * EPS)
    z[4, 0], z[4, 1], z[4, 2] = nan, inf, 1.0
    idx, w = route(z, 4)
    assert ftmoe.ftmoe_ops_status() == -10
    assert idx[4].tolist() == [2, -1, -1, -1] and w[4].tolist() == [1.0, 0.0, 0.0, 0.0]
    b = torch.zeros(8, device=DEV)
    b[7] = -inf
    idx, _ = route(z[3:4], 2, "sigmoid", bias=b)
    assert idx[0].tolist() == [6, 5] and ftmoe.ftmoe_ops_status() == 0
    b[7], b[6] = nan, inf
    idx, _ = route(z[3:4], 2, "sigmoid", bias=b)
    assert idx[0].tolist() == [5, 4] and ftmoe.ftmoe_ops_status() == -10


def test_route_strided_logits():
    g = gen(63)
    wide = randn(g, 20, 301)
    check_route(wide[:, 1:257], 8, "sigmoid", bias=randn(g, 256, std=0.1), groups=(8, 4, 2))


def route_grad_exact(logits, idx, scale, score, norm, dw):
    z = logits.double().requires_grad_()
    z0 = z.masked_fill(logits == -math.inf, -math.inf)
    p = torch.softmax(z0, 1) if score == "softmax" else torch.sigmoid(z0)
    at = idx.long().clamp(min=0)
    on = (idx >= 0).double()
    s = p.gather(1, at) * on
    w = scale * (s / s.sum(1, keepdim=True).clamp(min=1e-300) if norm else s)
    (w * dw.double()).sum().backward()
    return z.grad.nan_to_num(0.0)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups", ROUTES)
def test_route_backward(T, E, k, groups, score, norm):
    g = gen(64 + T + E)
    for dtype in (FP32, BF16):
        logits = randn(g, T, E, dtype=dtype, std=1.5)
        if E > k + 1 and groups[0] == 1:
            logits[0, 0] = -math.inf
        idx, w = route(logits, k, score, norm, 2.5, None, groups)
        dw = randn(g, T, k)
        exact = route_grad_exact(logits, idx, 2.5, score, norm, dw)
        new = Guarded()
        d = new((T, E), dtype)
        args = ftmoe.route_args(logits, idx, w, score=score, norm_topk_prob=norm, scale=2.5, n_groups=groups[0],
                                top_groups=groups[1], group_best=groups[2])
        ftmoe.ftmoe_route_topk_backward(args, dw, d)
        new.check()
        # terms are w u and w D: each within some 40 + k roundings of its size
        size = 2.5 * (dw.double().abs().amax(1, keepdim=True) * 2) + 0 * exact
        within(d, exact, UNIT[dtype] * exact.abs() + TINY[dtype] + (60 + k) * EPS * size)
        if dtype is FP32:  # in its input's place
            here = logits.clone()
            args = ftmoe.route_args(here, idx, w, score=score, norm_topk_prob=norm, scale=2.5, n_groups=groups[0],
                                    top_groups=groups[1], group_best=groups[2])
            ftmoe.ftmoe_route_topk_backward(args, dw, here)
            assert torch.equal(here, d)


def test_route_backward_against_differences():
    """d (sum dw w) / d logits by central differences of the forward's definition, the choice held."""
    g = gen(65)
    T, E, k = 4, 24, 5
    logits, dw = randn(g, T, E), randn(g, T, k)
    for score in ("softmax", "sigmoid"):
        for norm in (True, False):
            idx, w = route(logits, k, score, norm)
            d = torch.empty_like(logits)
            ftmoe.ftmoe_route_topk_backward(ftmoe.route_args(logits, idx, w, score=score, norm_topk_prob=norm), dw, d)
            step = 1e-4

            def f(z):
                p = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
                s = p.gather(1, idx.long())
                return ((s / s.sum(1, keepdim=True) if norm else s) * dw.double()).sum()

            for e in range(E):
                for t in range(T):
                    hi, lo = logits.double().clone(), logits.double().clone()
                    hi[t, e] += step
                    lo[t, e] -= step
                    slope = float((f(hi) - f(lo)) / (2 * step))
                    # the third derivative's term, step^2 times some |dw|, and fp32
                    assert abs(slope - float(d[t, e])) <= 1e-7 + 100 * EPS * float(dw[t].abs().sum())


def test_route_backward_equal_and_bad_indices():
    z = torch.zeros(1, 4, device=DEV)
    idx = torch.tensor([[2, 2, -1, 9]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.25, 0.25, 0.5, 0.5]], device=DEV)
    dw = torch.tensor([[1.0, 3.0, 5.0, 7.0]], device=DEV)
    d = torch.full((1, 4), 9.0, device=DEV)
    ftmoe.ftmoe_route_topk_backward(ftmoe.route_args(z, idx, w, score="sigmoid", norm_topk_prob=False), dw, d)
    assert ftmoe.ftmoe_ops_status() == -10
    assert d.tolist() == [[0.0, 0.0, 0.5, 0.0]]


def test_route_backward_into_strided_rows():
    """Only the rows' own values are written, wherever they start."""
    g = gen(67)
    logits, dw = randn(g, 9, 24, dtype=BF16), randn(g, 9, 3)
    idx, w = route(logits, 3, "sigmoid")
    want, wide = torch.empty_like(logits), torch.full((9, 33), 5.0, dtype=BF16, device=DEV)
    args = ftmoe.route_args(logits, idx, w, score="sigmoid")
    ftmoe.ftmoe_route_topk_backward(args, dw, want)
    ftmoe.ftmoe_route_topk_backward(args, dw, wide[:, 5:29])
    assert torch.equal(wide[:, 5:29], want)
    wide[:, 5:29] = 5.0
    assert bool((wide == 5.0).all())


# ----------------------------------------------------------------- sizes whose offsets pass 32 bits

def big_codes(g, *shape):
    """Random codes, NaN left out."""
    c = torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8)
    return torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.5, c | 128, c).view(E4M3)


def test_product_of_many_rows():
    """Rows times width beyond 2^31 values: the last rows are as a short call gives them."""
    g = gen(100)
    M, N, K = 600_000, 4096, 128
    a, a_scale = big_codes(g, M, K), torch.rand(1, M, generator=g, device=DEV)
    w, w_scale = bank(g, 1, N, K)
    out = torch.empty(M, N, dtype=BF16, device=DEV)
    ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, None, M, 1, N, K, out)
    few = torch.empty(100, N, dtype=BF16, device=DEV)
    for at in (0, 524_200, M - 100):
        ftmoe.ftmoe_fp8_matmul(a[at:at + 100].contiguous(), a_scale[:, at:at + 100].contiguous(), w, w_scale, None, 100, 1,
                               N, K, few)
        assert torch.equal(out[at:at + 100], few)


def test_product_of_the_most_rows():
    """M = 2^31 - 1, the largest count of rows."""
    g = gen(103)
    M, N, K = 2**31 - 1, 16, 16
    a, a_scale = torch.zeros(M, K, dtype=torch.uint8, device=DEV), torch.ones(1, M, device=DEV)
    w, w_scale = bank(g, 1, N, K)
    out, few = torch.full((M, N), 7.0, dtype=BF16, device=DEV), torch.empty(100, N, dtype=BF16, device=DEV)
    for at in (0, M - 100):
        a[at:at + 100] = big_codes(g, 100, K).view(torch.uint8)
    ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, None, M, 1, N, K, out)
    for at in (0, M - 100):
        ftmoe.ftmoe_fp8_matmul(a[at:at + 100], a_scale[:, at:at + 100].contiguous(), w, w_scale, None, 100, 1, N, K, few)
        assert torch.equal(out[at:at + 100], few)
    assert not bool(out[M // 2:M // 2 + 1000].any())


def test_product_with_a_large_bank():
    """Experts whose codes lie beyond 2^32 bytes."""
    g = gen(101)
    E, N, K = 72, 8192, 8192
    w, w_scale = big_codes(g, E, N, K), torch.rand(E, 64, 64, generator=g, device=DEV)
    a, a_scale = rows_of(g, 40, K)
    out, one = torch.empty(40, N, device=DEV), torch.empty(40, N, device=DEV)
    for e in (0, 63, 71):
        ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, offsets_of([0] * e + [40] + [0] * (E - 1 - e)), 40, E, N, K, out)
        ftmoe.ftmoe_fp8_matmul(a, a_scale, w[e], w_scale[e], None, 40, 1, N, K, one)
        assert torch.equal(out, one) and bool(out.isfinite().all())


def test_elementwise_calls_past_32_bits():
    g = gen(102)
    T, K = 290_000, 8192
    x = torch.randn(1000, K, generator=g, device=DEV).to(BF16).repeat(290, 1)
    codes, scales = torch.empty(T, K, dtype=E4M3, device=DEV), torch.empty(64, T, device=DEV)
    ftmoe.ftmoe_fp8_quantize(x, T, K, None, 1, codes, scales)
    want, scale = quantized(x[:1000])
    for at in (0, 262_000, T - 1000):
        same_codes(codes[at:at + 1000], want)
        assert torch.equal(scales[:, at:at + 1000], scale)
    h = torch.empty(T, K // 2, dtype=BF16, device=DEV)
    ftmoe.ftmoe_swiglu(x, T, K // 2, h)
    exact = silu_up(x[:1000])
    for at in (0, 262_000, T - 1000):
        within(h[at:at + 1000], exact, UNIT[BF16] * exact.abs() + TINY[BF16] + 8 * EPS * exact.abs())


# ----------------------------------------------------------------- together

def layer(g, T, H, I, E, k):
    w_gu, s_gu = bank(g, E, 2 * I, H, std=0.05)
    w_dn, s_dn = bank(g, E, H, I, std=0.05)
    return randn(g, T, H, dtype=BF16), randn(g, T, E), randn(g, E, std=0.05), (w_gu, s_gu), (w_dn, s_dn)


def forward(x, logits, bias, gu, dn, k, stream=None, keep=None):
    T, H = x.shape
    E, I = gu[0].shape[0], gu[0].shape[1] // 2
    P = T * k
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)
    f8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)
    f32 = lambda *s: torch.empty(*s, device=DEV)
    b = keep if keep is not None and keep else dict(
        idx=i32(T, k), w=f32(T, k), offsets=i32(E + 1), perm=i32(P), inv=i32(P), xs=f8(P, H), xs_s=f32(blocks(H), P),
        h=f8(P, I), h_s=f32(blocks(I), P), ys=torch.empty(P, H, dtype=BF16, device=DEV), out=torch.empty_like(x))
    if keep is not None:
        keep.update(b)
    ftmoe.ftmoe_route_topk(ftmoe.route_args(logits, b["idx"], b["w"], score="sigmoid", scale=2.0, bias=bias, n_groups=4,
                                            top_groups=2, group_best=2), stream=stream)
    ftmoe.ftmoe_dispatch(None, T, H, b["idx"], k, E, b["offsets"], b["perm"], b["inv"], None, stream=stream)
    ftmoe.ftmoe_fp8_quantize(x, T, H, b["inv"], k, b["xs"], b["xs_s"], stream=stream)
    ftmoe.ftmoe_fp8_matmul(b["xs"], b["xs_s"], *gu, b["offsets"], P, E, 2 * I, H, b["h"], b["h_s"], swiglu=True,
                           stream=stream)
    ftmoe.ftmoe_fp8_matmul(b["h"], b["h_s"], *dn, b["offsets"], P, E, H, I, b["ys"], stream=stream)
    ftmoe.ftmoe_combine(b["ys"], T, H, k, b["inv"], b["w"], b["out"], stream=stream)
    return b


@pytest.mark.parametrize("T", [1, 7, 200])
def test_layer_forward(T):
    """The whole layer against 64 bits.  A rounding to codes is off by an even spread of up to a 16th of the binade's
    start, 2^-5.4 of the values in the 2-norm.  x's passes through gate (SiLU's relative slope in the mean: up to 1.5)
    and up, h's comes on top, all independent from value to value: 2^-5.4 sqrt(1 + 1.5^2 + 1) = 0.049, held to 2^-4."""
    g = gen(70 + T)
    k = 4
    x, logits, bias, gu, dn = layer(g, T, 400, 256, 16, k)
    b = forward(x, logits, bias, gu, dn, k)
    want, ww, near = routed(logits, k, "sigmoid", True, 2.0, bias, (4, 2, 2))
    assert np.array_equal(b["idx"].cpu().numpy(), want)
    wg, wd = bank_value(*gu), bank_value(*dn)
    y = torch.zeros(T, 400, dtype=torch.float64, device=DEV)
    for t in range(T):
        for j in range(k):
            e = int(want[t, j])
            y[t] += float(ww[t, j]) * (wd[e] @ silu_up((wg[e] @ x[t].double())[None])[0])
    assert float((b["out"].double() - y).norm() / y.norm()) <= 2.0 ** -4


def test_layer_captured_and_on_streams():
    """Captured once and replayed on new inputs, and on two streams at once, the layer gives the direct call's bits."""
    g = gen(80)
    k, T = 4, 50
    x, logits, bias, gu, dn = layer(g, T, 400, 256, 16, k)
    x2, logits2 = randn(g, T, 400, dtype=BF16), randn(g, T, 16)
    one = forward(x, logits, bias, gu, dn, k)["out"].clone()
    two = forward(x2, logits2, bias, gu, dn, k)["out"].clone()
    xin, lin, keep = x.clone(), logits.clone(), {}
    forward(xin, lin, bias, gu, dn, k, keep=keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(xin, lin, bias, gu, dn, k, keep=keep)
    for a, l, want in ((x2, logits2, two), (x, logits, one), (x2, logits2, two)):
        xin.copy_(a)
        lin.copy_(l)
        keep["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(keep["out"], want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [forward(a, l, bias, gu, dn, k, stream=s) for s, (a, l) in zip(streams * 3, [(x, logits), (x2, logits2)] * 3)]
    torch.cuda.synchronize()
    for b, want in zip(got, [one, two] * 3):
        assert torch.equal(b["out"], want)


def test_layer_backward():
    """The gradients of tokens and logits through the layer against automatic differentiation in 64 bits.  Roundings to
    codes, 2^-5.4 each in the 2-norm (see the forward pass), enter by dys, by x through gate and up (slopes up to 1.5
    and 1) and by dgu, and bf16's are small beside them: 2^-5.4 sqrt(1 + 1.5^2 + 1 + 1) = 0.054 for dx, and the
    forward's 0.049 for dw, of which the router takes differences (twice that): the 2-norms are held to 2^-3."""
    g = gen(90)
    T, H, I, E, k = 60, 400, 256, 16, 4
    x, logits, bias, gu, dn = layer(g, T, H, I, E, k)
    P = T * k
    b = forward(x, logits, bias, gu, dn, k)
    new16 = lambda *s: torch.empty(*s, dtype=BF16, device=DEV)
    gu_rows, h, h_s = new16(P, 2 * I), torch.empty(P, I, dtype=E4M3, device=DEV), torch.empty(2, P, device=DEV)
    ftmoe.ftmoe_fp8_matmul(b["xs"], b["xs_s"], *gu, b["offsets"], P, E, 2 * I, H, gu_rows)
    ftmoe.ftmoe_swiglu(gu_rows, P, I, h, h_s, used=b["offsets"][E:])
    ys = new16(P, H)
    ftmoe.ftmoe_fp8_matmul(h, h_s, *dn, b["offsets"], P, E, H, I, ys)
    dout = randn(g, T, H, dtype=BF16)
    dys, dw = new16(P, H), torch.empty(T, k, device=DEV)
    ftmoe.ftmoe_combine_backward(dout, ys, T, H, k, b["inv"], b["w"], dys, dw)
    q, q_s = torch.empty(P, H, dtype=E4M3, device=DEV), torch.empty(blocks(H), P, device=DEV)
    ftmoe.ftmoe_fp8_quantize(dys, P, H, None, 1, q, q_s, used=b["offsets"][E:])
    dh = new16(P, I)
    ftmoe.ftmoe_fp8_matmul(q, q_s, *dn, b["offsets"], P, E, H, I, dh, transpose=True)
    dgu, dgu_s = torch.empty(P, 2 * I, dtype=E4M3, device=DEV), torch.empty(4, P, device=DEV)
    ftmoe.ftmoe_swiglu_backward(dh, gu_rows, P, I, dgu, dgu_s, used=b["offsets"][E:])
    dxs, dx = new16(P, H), new16(T, H)
    ftmoe.ftmoe_fp8_matmul(dgu, dgu_s, *gu, b["offsets"], P, E, 2 * I, H, dxs, transpose=True)
    ftmoe.ftmoe_combine(dxs, T, H, k, b["inv"], None, dx)
    dl = torch.empty_like(logits)
    args = ftmoe.route_args(logits, b["idx"], b["w"], score="sigmoid", scale=2.0, bias=bias, n_groups=4, top_groups=2,
                            group_best=2)
    ftmoe.ftmoe_route_topk_backward(args, dw, dl)
    xv, z = x.double().requires_grad_(), logits.double().requires_grad_()
    s = torch.sigmoid(z).gather(1, b["idx"].long())
    w = 2.0 * s / s.sum(1, keepdim=True)
    wg, wd = bank_value(*gu), bank_value(*dn)
    y = 0
    for j in range(k):
        e = b["idx"][:, j].long()
        gate, up = torch.einsum("th,tnh->tn", xv, wg[e]).chunk(2, 1)
        y = y + w[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(gate) * up, wd[e])
    (y * dout.double()).sum().backward()
    assert float((dx.double() - xv.grad).norm() / xv.grad.norm()) <= 2.0 ** -3
    assert float((dl.double() - z.grad).norm() / z.grad.norm()) <= 2.0 ** -3
