"""The layer on 8-bit codes where its calls give up, or where their arithmetic has least to spare.  Bounds are those
of the layer's other tests: EPS is half a step of fp32, 2^-24."""

import pytest
import torch

from nvfp4_mixture_experts_counting_gb300 import ftmoe

from test_gpu_fp8_layer import CODE, CODE_TINY, E4M3, bank, offsets_of, product, rows_of, value
from test_gpu_train_ops import BF16, DEV, EPS, FP32, TINY, UNIT, Guarded, built, gen, within  # noqa: F401

pytestmark = pytest.mark.gpu
FORMS = pytest.mark.parametrize("form", ["plain", "transpose", "swiglu"])


# ----------------------------------------------------------------- a wait that runs out

def call_product(a, a_scale, w, w_scale, counts, form, dtype=BF16):
    """Outputs between guards (codes and scales with SwiGLU), their bytes 9 and scales 5.0 beforehand; `counts` of each
    expert, or the offsets."""
    new, M, (E, N, K) = Guarded(), a.shape[0], w.shape
    O = K if form == "transpose" else N // 2 if form == "swiglu" else N
    out = new((M, O), E4M3 if form == "swiglu" else dtype)
    out.view(torch.uint8).fill_(9)
    scales = new((O // 128, M), FP32, 5.0) if form == "swiglu" else None
    offsets = counts if torch.is_tensor(counts) else offsets_of(counts)
    ftmoe.ftmoe_fp8_matmul(a, a_scale, w, w_scale, offsets, M, E, N, K, out, scales,
                           transpose=form == "transpose", swiglu=form == "swiglu")
    new.check()
    return out, scales


def first_ctas_tiles(M, O, counts, form):
    """(rows, columns) of the tiles that the first CTA has: an expert's tiles in order, 128 rows by 256 columns (128 of
    h), rows fastest; a CTA takes every one of as many as there are SMs, or could be tiles."""
    width = 128 if form == "swiglu" else 256
    columns = -(-O // width)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    grid = min((M // 128 + min(M, len(counts))) * columns, sms)
    units, at = [], 0
    for n in counts:
        units += [(slice(at + r, at + min(n, r + 128)), slice(j * width, min(O, (j + 1) * width)))
                  for j in range(columns) for r in range(0, n, 128)]
        at += n
    return units[::grid]


@FORMS
@pytest.mark.parametrize("counts,N,K", [
    ([2, 0, 3], 256, 144), ([1], 256, 16),           # a tile or two of one block or two
    ([700, 0, 300], 1280, 640), ([129, 1, 0, 127, 43], 256, 2000),
    ([2500, 0, 4000, 1500, 333], 1280, 1040)])       # the first CTA has several tiles
def test_product_wait_that_runs_out(counts, N, K, form):
    """The first CTA's first tokens are never asked for: its waits end after 2 ms each, the call reports it and leaves
    that CTA's tiles, the others are as they should be, and the next call is as good as new."""
    g, M, E = gen(110 + N + K + len(counts)), sum(counts), len(counts)
    a, a_scale = rows_of(g, M, N if form == "transpose" else K)
    w, w_scale = bank(g, E, N, K)
    want, want_scale = call_product(a, a_scale, w, w_scale, counts, form)
    assert ftmoe.ftmoe_ops_status() == 0
    ftmoe.ftmoe_test_withhold_matmul(True, 2_000_000)
    try:
        got, got_scale = call_product(a, a_scale, w, w_scale, counts, form)
    finally:
        ftmoe.ftmoe_test_withhold_matmul(False)
    assert ftmoe.ftmoe_ops_status() == -7 and ftmoe.ftmoe_ops_status() == 0
    again, again_scale = call_product(a, a_scale, w, w_scale, counts, form)
    assert ftmoe.ftmoe_ops_status() == 0
    assert torch.equal(again.view(torch.uint8), want.view(torch.uint8))
    for rows, cols in first_ctas_tiles(M, want.shape[1], counts, form):
        size = want.element_size()
        want.view(torch.uint8).view(M, -1)[rows, cols.start * size:cols.stop * size] = 9
        if form == "swiglu":
            want_scale[cols.start // 128, rows] = 5.0
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    if form == "swiglu":
        assert torch.equal(got_scale, want_scale)


# ----------------------------------------------------------------- SwiGLU of far negative gates

@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_swiglu_of_far_negative_gates(dtype):
    """Sigmoids next to fp32's smallest numbers times large factors.  exp is within two of fp32's last places, which
    are 2^-149 there, and its product with the reciprocal adds half of one: sigmoid is within 2.5 2^-149, SiLU's
    rounding adds 2^-150; all else is relative as for other gates."""
    I, big = 128, 2.0 ** 50
    g = torch.linspace(-104.0, -80.0, 64 * I, device=DEV).view(64, I).to(dtype)
    gu = torch.cat([g, torch.full_like(g, big)], 1)
    dh = torch.full_like(g, big)
    z, s = g.double(), torch.sigmoid(g.double())
    exact, unit, last = z * s * big, UNIT[dtype], 2.5 * 2.0 ** -149
    bound = (last * z.abs() + 2.0 ** -150) * big + 8 * EPS * exact.abs()
    new = Guarded()
    h, dgu = new((64, I), dtype), new((64, 2 * I), dtype)
    ftmoe.ftmoe_swiglu(gu, 64, I, h)
    within(h, exact, bound * (1 + unit) + unit * exact.abs())
    codes, scales = new((64, I), E4M3), new((1, 64), FP32)
    ftmoe.ftmoe_swiglu(gu, 64, I, codes, scales)
    top = exact.abs().amax(1)
    within(scales[0], top / 448, (bound.amax(1) + 2 * EPS * top) / 448)
    ftmoe.ftmoe_swiglu_backward(dh, gu, 64, I, dgu)
    dg, du = big * big * s * (1 + z * (1 - s)), big * z * s
    rel = 2.0 ** -20
    dg_bound = big * big * (1 + z.abs()) * (last + rel * s)
    du_bound = big * z.abs() * (last + rel * s)
    within(dgu[:, :I], dg, dg_bound * (1 + unit) + unit * dg.abs())
    within(dgu[:, I:], du, du_bound * (1 + unit) + unit * du.abs())
    new.check()


# ----------------------------------------------------------------- routing

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [1.0, 2.5, 0.1, 1.7, 3.3])
def test_route_equal_weights_round_once(scale, score):
    """n equal logits: scores are 1 (or 1/2), their sum n (or n/2), all exact, so that a weight is scale / n rounded."""
    k, E = 32, 64
    logits = torch.full((k, E), -float("inf"), device=DEV)
    for n in range(1, k + 1):
        logits[n - 1, :n] = 0.0
    new = Guarded()
    idx, w = new((k, k), torch.int32), new((k, k), FP32)
    ftmoe.ftmoe_route_topk(ftmoe.route_args(logits, idx, w, score=score, scale=scale))
    new.check()
    at = torch.arange(k, device=DEV)
    on = at[None] <= at[:, None]
    want = torch.full((k, k), scale, device=DEV) / (at + 1.0)[:, None]
    assert torch.equal(w, torch.where(on, want, 0.0))
    assert torch.equal(idx, torch.where(on, at[None], -1).int())


def test_route_reads_the_biases_that_the_previous_kernel_wrote():
    """Biases change between calls in a row, in the stream and in a graph (the call starts while the copy ends)."""
    g = gen(120)
    T, E, k, n = 64, 256, 8, 6
    logits, biases = torch.randn(T, E, generator=g, device=DEV), torch.randn(n, E, generator=g, device=DEV)
    bias, idx = torch.zeros(E, device=DEV), torch.empty(n, T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(n, T, k, device=DEV)
    args = [ftmoe.route_args(logits, idx[i], w[i], score="sigmoid", bias=bias) for i in range(n)]
    for i in range(n):
        bias.copy_(biases[i])
        torch.cuda.synchronize()
        ftmoe.ftmoe_route_topk(args[i])
        torch.cuda.synchronize()
    want, want_w = idx.clone(), w.clone()

    def pass_():
        for i in range(n):
            bias.copy_(biases[i])
            ftmoe.ftmoe_route_topk(args[i])

    def same():
        torch.cuda.synchronize()
        ok = torch.equal(idx, want) and torch.equal(w, want_w)
        idx.fill_(-9)
        return ok

    assert not torch.equal(want[0], want[1])
    idx.fill_(-9)
    for _ in range(50):
        pass_()
        assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pass_()
    for _ in range(50):
        graph.replay()
        assert same()


# ----------------------------------------------------------------- the product's scales and its SwiGLU

def test_product_swiglu_of_all_gates():
    """Rows whose gate is one number and whose up is its magnitude times 2^60, so that their scale is |h| / 448 and
    shows h's error: (1.25 |g| + 8) of SiLU, the product with up and the scale's rounding; 0 below -87.3."""
    n, I, K = 1 << 14, 128, 16
    size = torch.linspace(0.005, 87.3, n, device=DEV)
    a, a_scale = torch.zeros(2 * n + 64, K, device=DEV), torch.empty(1, 2 * n + 64, device=DEV)
    a[:, 0], a[:, 1] = -1.0, 1.0
    a[:n, 0] = 1.0
    a_scale[0] = torch.cat([size, size, torch.linspace(87.4, 300.0, 64, device=DEV)])
    w, w_scale = torch.zeros(1, 2 * I, K, device=DEV), torch.tensor([[[1.0], [2.0 ** 60]]], device=DEV)
    w[0, :I, 0] = 1.0
    w[0, I:, 1] = 1.0
    _, scales = call_product(a.to(E4M3), a_scale, w.to(E4M3), w_scale, [2 * n + 64], "swiglu")
    g = torch.cat([size, -size]).double()
    h = g * torch.sigmoid(g) * g.abs() * 2.0 ** 60
    within(scales[0, :2 * n], h.abs() / 448, (1.25 * g.abs() + 10) * EPS * h.abs() / 448 * (1 + 2.0 ** -16))
    assert bool((scales[0, 2 * n:] == 0).all())


@pytest.mark.parametrize("form", ["plain", "transpose"])
@pytest.mark.parametrize("of_rows,of_weights", [(-120, -6), (-6, -120), (120, -120), (-120, 120), (100, 20), (20, 100)])
def test_product_of_far_scales(of_rows, of_weights, form):
    """Scales are powers of two whose product fp32 holds; small whole codes, so that every sum is exact."""
    g = gen(130)
    M, N, K = 150, 272, 400
    C = N if form == "transpose" else K
    q = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV).float()
    x, m = q(M, C), q(1, N, K)
    a_scale = torch.full((-(-C // 128), M), 2.0 ** of_rows, device=DEV)
    w_scale = torch.full((1, -(-N // 128), -(-K // 128)), 2.0 ** of_weights, device=DEV)
    out, _ = call_product(x.to(E4M3), a_scale, m.to(E4M3), w_scale, [M], form, FP32)
    y = x.double() @ (m[0] if form == "transpose" else m[0].t()).double()
    assert torch.equal(out.double(), y * 2.0 ** (of_rows + of_weights))


# ----------------------------------------------------------------- the product's units and offsets

MANY = [2555, 0, 4011, 1533, 3901]  # copies of 128 tokens, several units a CTA, ragged last tiles


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("C", [272, 512, 1040])
@pytest.mark.parametrize("transpose", [False, True])
def test_product_of_many_tokens_an_expert(transpose, C, dtype):
    g, M, O = gen(140 + C), sum(MANY), 1280
    N, K = (C, O) if transpose else (O, C)
    a, a_scale = rows_of(g, M, C)
    w, w_scale = bank(g, len(MANY), N, K)
    y, bound = product(a, a_scale, w, w_scale, MANY, transpose)
    form, unit = "transpose" if transpose else "plain", 0.0 if dtype is FP32 else UNIT[dtype]
    first, _ = call_product(a, a_scale, w, w_scale, MANY, form, dtype)
    within(first, y, bound * (1 + unit) + unit * y.abs() + TINY[dtype])
    for _ in range(3):
        assert torch.equal(call_product(a, a_scale, w, w_scale, MANY, form, dtype)[0], first)


@pytest.mark.parametrize("K", [272, 512, 1040])
def test_product_with_swiglu_of_many_tokens_an_expert(K):
    g, M, I = gen(150 + K), sum(MANY), 640
    a, a_scale = rows_of(g, M, K)
    w, w_scale = bank(g, len(MANY), 2 * I, K, std=0.1)
    y, bound = product(a, a_scale, w, w_scale, MANY, False)
    gate, up = y.chunk(2, 1)
    dg, du = bound.chunk(2, 1)
    h = gate * torch.sigmoid(gate) * up
    # |d SiLU| <= 1.1; SiLU's own error, and the product's
    err = 1.1 * dg * (up.abs() + du) + (gate * torch.sigmoid(gate)).abs() * du + (1.25 * gate.abs() + 9) * EPS * h.abs()
    worst, top = (v.view(M, -1, 128).amax(2) for v in (err, h.abs()))
    first, scales = call_product(a, a_scale, w, w_scale, MANY, "swiglu")
    within(scales.t(), top / 448, (worst + 2 * EPS * top) / 448 + 1e-30)
    wide, spread = (v.repeat_interleave(128, 1) for v in (top / 448, worst))
    within(value(first, scales), h,
           (CODE * h.abs() + CODE_TINY * wide) * (1 + 2.0 ** -16) + 2 * err + 2 * spread + 1e-30)
    for _ in range(3):
        again, again_scales = call_product(a, a_scale, w, w_scale, MANY, "swiglu")
        assert torch.equal(again.view(torch.uint8), first.view(torch.uint8)) and torch.equal(again_scales, scales)


BIG = 2 ** 31 - 1
TABLES = [
    [0, 5, 10, 9, 20], [0, 5, 10, 21, 20], [0, 5, 10, -4, 20], [0, 5, 10, 1 << 30, -(1 << 30)], [0, 5, 4, 10, 20],
    [3, 5, 10, 15, 21], [-1, 5, 10, 15, 20], [BIG, 5, 10, 15, 20], [0, BIG, 10, 15, 20], [0, 0, 20, 0, 20],
    [5, 4, 3, 2, 1], [-BIG - 1, BIG, -BIG - 1, BIG, 20]]


@FORMS
@pytest.mark.parametrize("table", TABLES, ids=str)
def test_product_leaves_out_bad_experts_alone(table, form):
    """Only the rows of experts that the header calls good are written, and each as it would be by itself."""
    g, M, E, N, K = gen(160), 20, 4, 256, 128
    a, a_scale = rows_of(g, M, N if form == "transpose" else K)
    w, w_scale = bank(g, E, N, K)
    alone = [call_product(a, a_scale, w[e:e + 1], w_scale[e:e + 1], [M], form) for e in range(E)]
    offsets = torch.tensor(table, dtype=torch.int32, device=DEV)
    got, scales = call_product(a, a_scale, w, w_scale, offsets, form)
    want = torch.full_like(got.view(torch.uint8), 9)
    want_scales = None if scales is None else torch.full_like(scales, 5.0)
    bad = False
    for e in range(E):
        lo, hi = table[e], table[e + 1]
        if not max([0] + table[:e + 1]) <= lo <= hi <= M:
            bad = True
            continue
        want[lo:hi] = alone[e][0].view(torch.uint8)[lo:hi]
        if scales is not None:
            want_scales[:, lo:hi] = alone[e][1][:, lo:hi]
    assert bad and ftmoe.ftmoe_ops_status() == -10
    assert torch.equal(got.view(torch.uint8), want)
    assert scales is None or torch.equal(scales, want_scales)
