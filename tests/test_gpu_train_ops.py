"""The training operators against their definitions in 64 bits, at the sizes
and masks where they can go wrong.

Bounds.  A value computed in fp32 and rounded once to its type is within
u |v| of the exact one plus the fp32 error, u the type's unit roundoff (half
an ulp, relative) and, below the type's normal range, half its smallest
subnormal.  A sum of n terms in fp32 in any order is within
(n + 2) 2^-24 sum |terms| of the exact one to first order; the bounds below
double that.  Every output lies between guard values, so a write out of
range shows."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

from nvfp4_mixture_experts_counting_gb300 import ftmoe, workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
UNIT = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -126}  # fp32 subnormals may flush
NAMES = {BF16: "bf16", FP16: "fp16", FP32: "fp32"}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from nvfp4_mixture_experts_counting_gb300 import build
    build.build()
    ftmoe.ftmoe_ops_status()
    yield
    assert ftmoe.ftmoe_ops_status() == 0  # every test that marks the word reads it


class Guarded:
    """Outputs with 64 guard values on both sides of each."""

    def __init__(self):
        self.kept = []

    def __call__(self, shape, dtype, fill=None):
        n = int(np.prod(shape)) if shape else 1
        size = torch.tensor([], dtype=dtype).element_size()
        pad = 256 // size
        raw = torch.empty(pad + n + pad, dtype=dtype, device=DEV)
        raw.view(torch.uint8).fill_(0x55)
        self.kept.append((raw, pad, n))
        out = raw[pad:pad + n].view(shape)
        if fill is not None:
            out.fill_(fill)
        return out

    def check(self):
        for raw, pad, n in self.kept:
            b, size = raw.view(torch.uint8), raw.element_size()
            assert bool((b[:pad * size] == 0x55).all()) and bool((b[(pad + n) * size:] == 0x55).all())


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=FP32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def within(got, exact, bound):
    got, exact = got.double().cpu(), torch.as_tensor(exact).cpu()
    over = (got - exact).abs() - torch.as_tensor(bound).cpu()
    assert bool((over <= 0).all()), float(over.max())


def choose(g, T, k, E, drop=0.0):
    """Distinct experts per token, some dropped; the first token loses all when any may be dropped."""
    idx = torch.argsort(torch.rand(T, E, generator=g, device=DEV), 1)[:, :k].int().contiguous()
    if drop and T:
        idx[torch.rand(T, k, generator=g, device=DEV) < drop] = -1
        idx[0] = -1
    return idx


def tables(idx, E):
    """offsets, perm and inv from the definition, on the host."""
    e = idx.cpu().numpy().reshape(-1)
    keep = (e >= 0) & (e < E)
    order = sorted((int(e[p]), p) for p in range(len(e)) if keep[p])
    offsets = np.array([sum(1 for x, _ in order if x < b) for b in range(E + 1)]) if len(order) * E < 1 << 18 else \
        np.searchsorted([x for x, _ in order], np.arange(E + 1))
    perm, inv = np.full(len(e), -1), np.full(len(e), -1)
    for at, (_, p) in enumerate(order):
        perm[at], inv[p] = p, at
    return offsets, perm, inv


def dispatch(idx, E, x=None, fill=7.0, stream=None):
    T, k = idx.shape
    new = Guarded()
    H = x.shape[1] if x is not None else 1
    off, perm, inv = new((E + 1,), torch.int32), new((T * k,), torch.int32), new((T * k,), torch.int32)
    xs = new((T * k, H), x.dtype, fill) if x is not None else None
    ftmoe.ftmoe_dispatch(x, T, H, idx, k, E, off, perm, inv, xs, stream=stream)
    torch.cuda.synchronize()
    new.check()
    return off, perm, inv, xs


# ----------------------------------------------------------------- tokens by expert

@pytest.mark.parametrize("T,k,E,H,dtype,drop", [
    (0, 2, 5, 16, BF16, 0.0), (1, 1, 1, 1, FP32, 0.0), (1, 8, 256, 2560, BF16, 0.0), (5, 3, 7, 33, BF16, 0.3),
    (16, 8, 256, 2560, BF16, 0.0), (77, 6, 60, 1001, FP16, 0.25), (128, 32, 1024, 24, FP32, 0.5),
    (512, 8, 9, 40, BF16, 0.1),           # the last size that counts in one launch
    (513, 8, 256, 80, BF16, 0.0),         # the first that sorts
    (1029, 4, 1024, 6, FP32, 0.3), (700, 32, 33, 17, FP16, 0.9), (9000, 1, 2, 4, BF16, 0.2)])
def test_dispatch(T, k, E, H, dtype, drop):
    g = gen(T * 31 + H)
    idx, x = choose(g, T, k, E, drop), randn(g, T, H, dtype=dtype)
    off, perm, inv, xs = dispatch(idx, E, x)
    o, p, i = tables(idx, E)
    assert np.array_equal(off.cpu(), o) and np.array_equal(perm.cpu(), p) and np.array_equal(inv.cpu(), i)
    kept = int(o[-1])
    token = torch.from_numpy(p[:kept] // k).to(DEV)
    assert torch.equal(xs[:kept], x[token]) and bool((xs[kept:] == 7.0).all())
    # the tables alone
    for a, b in zip(dispatch(idx, E)[:3], (off, perm, inv)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 2000])
def test_dispatch_all_dropped_and_all_on_one_expert(T):
    x = randn(gen(T), T, 8, dtype=BF16)
    off, perm, inv, xs = dispatch(torch.full((T, 4), -1, dtype=torch.int32, device=DEV), 6, x)
    assert not off.any() and bool((perm == -1).all()) and bool((inv == -1).all()) and bool((xs == 7.0).all())
    off, perm, inv, xs = dispatch(torch.full((T, 4), 5, dtype=torch.int32, device=DEV), 6, x)
    assert off.tolist() == [0, 0, 0, 0, 0, 0, 4 * T]
    assert torch.equal(perm, torch.arange(4 * T, device=DEV, dtype=torch.int32)) and torch.equal(perm, inv)
    assert torch.equal(xs, x.repeat_interleave(4, 0))


@pytest.mark.parametrize("T", [4, 3000])
def test_dispatch_marks_experts_out_of_range(T):
    idx = choose(gen(1), T, 2, 8)
    assert ftmoe.ftmoe_ops_status() == 0
    idx[T - 1, 1] = 8
    idx[0, 0] = -5  # dropped without a mark
    off, perm, inv, _ = dispatch(idx, 8)
    o, p, i = tables(idx, 8)
    assert np.array_equal(off.cpu(), o) and np.array_equal(perm.cpu(), p) and np.array_equal(inv.cpu(), i)
    assert ftmoe.ftmoe_ops_status() == -10 and ftmoe.ftmoe_ops_status() == 0


def test_dispatch_gives_the_layer_routing_tables():
    wl = W.WORKLOADS["tiny"]
    T, k, E = 60, wl.top_k, wl.E
    x, rw = randn(gen(3), T, wl.H, dtype=BF16), W.router_weight(wl, device=DEV)
    new = lambda *s, d=torch.int32: torch.empty(*s, dtype=d, device=DEV)
    idx, w, off, perm, inv = new(T, k), new(T, k, d=FP32), new(E + 1), new(T * k), new(T * k)
    ftmoe.ftmoe_route_static(x, T, wl.H, rw, None, E, k, True, idx, w, off, perm, inv)
    for a, b in zip(dispatch(idx, E)[:3], (off, perm, inv)):
        assert torch.equal(a, b)


PAIRS = [(1, 1, 1, 1, FP32, 0.0), (1, 8, 256, 2560, BF16, 0.0), (3, 5, 9, 33, BF16, 0.4), (64, 8, 32, 1024, FP16, 0.0),
         (77, 9, 60, 1001, FP16, 0.25), (40, 32, 64, 130, FP32, 0.5), (2500, 2, 7, 16, BF16, 0.3), (33, 17, 40, 8, FP32, 0.9)]


@pytest.mark.parametrize("T,k,E,H,dtype,drop", PAIRS)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, E, H, dtype, drop, weighted):
    g = gen(T + 7 * H)
    _, _, inv, _ = dispatch(choose(g, T, k, E, drop), E)
    ys, w = randn(g, T * k, H, dtype=dtype), torch.rand(T, k, generator=g, device=DEV)
    kept = int((inv >= 0).sum())
    ys[kept:] = float("nan")  # rows of no pair are not read
    new = Guarded()
    out = new((T, H), dtype)
    ftmoe.ftmoe_combine(ys, T, H, k, inv, w if weighted else None, out)
    torch.cuda.synchronize()
    new.check()
    i = inv.view(T, k).long()
    terms = ys[i.clamp(min=0)].double() * (w.double() if weighted else torch.ones_like(w).double())[:, :, None]
    terms = torch.where((i >= 0)[:, :, None], terms, 0.0)
    ref = terms.sum(1)
    within(out, ref, UNIT[dtype] * ref.abs() * 1.01 + 2 * (k + 2) * EPS * terms.abs().sum(1) + TINY[dtype])


@pytest.mark.parametrize("T,k,E,H,dtype,drop", PAIRS)
@pytest.mark.parametrize("in_place", [False, True])
def test_combine_backward(T, k, E, H, dtype, drop, in_place):
    g = gen(T + 11 * H)
    _, _, inv, _ = dispatch(choose(g, T, k, E, drop), E)
    P = T * k
    new = Guarded()
    ys, dout, w = new((P, H), dtype), randn(g, T, H, dtype=dtype), torch.rand(T, k, generator=g, device=DEV)
    ys.copy_(randn(g, P, H, dtype=dtype))
    before = ys.clone()
    dys = ys if in_place else new((P, H), dtype, 7.0)
    dw = new((T, k), FP32)
    ftmoe.ftmoe_combine_backward(dout, ys, T, H, k, inv, w, dys, dw)
    torch.cuda.synchronize()
    new.check()
    i = inv.view(T, k).long()
    kept = int((inv >= 0).sum())
    assert torch.equal(dys[kept:], before[kept:]) if in_place else bool((dys[kept:] == 7.0).all())
    for j in range(k):
        on = i[:, j] >= 0
        ref = w[on, j:j + 1].double() * dout[on].double()
        within(dys[i[on, j]], ref, UNIT[dtype] * ref.abs() * 1.01 + TINY[dtype])
        terms = torch.where(on[:, None], before[i[:, j].clamp(min=0)].double() * dout.double(), 0.0)
        within(dw[:, j], terms.sum(1), 2 * (H + 2) * EPS * terms.abs().sum(1))


def test_places_out_of_range_are_dropped_and_marked():
    T, k, H = 9, 2, 32
    _, _, inv, _ = dispatch(choose(gen(2), T, k, 5), 5)
    ys, w, out = randn(gen(3), T * k, H), torch.ones(T, k, device=DEV), torch.empty(T, H, device=DEV)
    bad = inv.clone()
    bad[3], bad[8] = T * k, -2
    good = inv.clone()
    good[3] = good[8] = -1
    ref, dys, dw = out.clone(), torch.zeros_like(ys), torch.empty(T, k, device=DEV)
    ftmoe.ftmoe_combine(ys, T, H, k, good, w, ref)
    assert ftmoe.ftmoe_ops_status() == 0
    ftmoe.ftmoe_combine(ys, T, H, k, bad, w, out)
    assert ftmoe.ftmoe_ops_status() == -10 and torch.equal(out, ref)
    ftmoe.ftmoe_combine_backward(ref, ys, T, H, k, bad, w, dys, dw)
    assert ftmoe.ftmoe_ops_status() == -10 and float(dw.view(-1)[3]) == 0.0 and float(dw.view(-1)[8]) == 0.0


def test_dispatch_and_combine_are_adjoint():
    """<dispatch(x), y> = <x, combine(y)> and <combine(y), d> = <y, combine_backward(d)>."""
    T, k, E, H = 37, 4, 12, 100
    g = gen(8)
    idx, x, d = choose(g, T, k, E, 0.2), randn(g, T, H), randn(g, T, H)
    _, _, inv, xs = dispatch(idx, E, x, fill=0.0)
    y, w = randn(g, T * k, H), torch.rand(T, k, generator=g, device=DEV)
    y[int((inv >= 0).sum()):] = 0.0
    back, out = torch.empty(T, H, device=DEV), torch.empty(T, H, device=DEV)
    ftmoe.ftmoe_combine(y, T, H, k, inv, None, back)
    ftmoe.ftmoe_combine(y, T, H, k, inv, w, out)
    dys, dw = torch.zeros_like(y), torch.empty(T, k, device=DEV)
    ftmoe.ftmoe_combine_backward(d, y, T, H, k, inv, w, dys, dw)
    dot = lambda a, b: float((a.double() * b.double()).sum())
    size = float((xs.double() * y.double()).abs().sum())
    assert abs(dot(xs, y) - dot(x, back)) <= 2 * (k + 2) * EPS * size
    size = float((dys.double() * y.double()).abs().sum())
    assert abs(dot(out, d) - dot(y, dys)) <= 2 * (k + 3) * EPS * size
    assert abs(dot(out, d) - dot(w, dw)) <= 2 * (k + H + 4) * EPS * size


@pytest.mark.parametrize("T,k,E,norm", [(1, 1, 1, True), (1, 1, 1, False), (5, 3, 7, True), (5, 3, 7, False),
                                        (33, 8, 256, True), (33, 8, 256, False), (9, 32, 1000, True), (9, 32, 1000, False)])
def test_route_backward(T, k, E, norm):
    g = gen(T + E)
    z = (torch.randn(T, E, generator=g, device=DEV) * 3)
    if E > 7 and not norm:
        z[0, :E // 2] = -float("inf")  # experts that a mask took out
    top, idx = torch.topk(z, k, dim=1)
    idx = idx.int().contiguous()
    w = (torch.softmax(top, 1) if norm else torch.softmax(z, 1).gather(1, idx.long())).contiguous()
    dw = randn(g, T, k)
    new = Guarded()
    out = new((T, E), FP32)
    ftmoe.ftmoe_route_backward(None if norm else z, idx, w, dw, T, E, k, norm, out)
    torch.cuda.synchronize()
    new.check()
    # the formula, against 64-bit automatic differentiation of the weights
    z64 = z.double().requires_grad_()
    if norm:
        w64 = torch.softmax(z64.gather(1, idx.long()), 1)
    else:
        w64 = torch.softmax(z64, 1).gather(1, idx.long())
    (w64 * dw.double()).sum().backward()
    ref = z64.grad
    spread = float((z - z.amax(1, keepdim=True))[torch.isfinite(z)].abs().max())
    rel = 2 * EPS * (64 + E / 32 + spread)  # exponential, its argument, sums over k and over E
    prob = torch.softmax(z64.detach(), 1) if not norm else torch.zeros_like(ref).scatter_(1, idx.long(), w64.detach())
    total = (w64.detach() * dw.double().abs()).sum(1, keepdim=True)
    mine = torch.zeros_like(ref).scatter_(1, idx.long(), dw.double().abs())
    within(out, ref, rel * prob * (mine + total))


def test_route_backward_marks_and_skips_bad_indices():
    idx = torch.tensor([[0, 9], [2, -1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, 0.5], [0.25, 0.75]], device=DEV)
    dw, out = torch.tensor([[1.0, 3.0], [2.0, 0.0]], device=DEV), torch.empty(2, 4, device=DEV)
    ftmoe.ftmoe_route_backward(None, idx, w, dw, 2, 4, 2, True, out)
    assert ftmoe.ftmoe_ops_status() == -10
    # S = 2 and 0.5: w (dw - S) at the valid slots only
    assert out.tolist() == [[-0.5, 0.0, 0.0, 0.0], [0.0, 0.0, 0.375, 0.0]]


# ----------------------------------------------------------------- embedding

def token_ids(g, N, V, kind):
    if kind == "one":
        return torch.full((N,), V // 2, device=DEV)
    if kind == "few":  # runs of many lengths
        return (torch.rand(N, generator=g, device=DEV) ** 3 * min(V, 9)).long()
    return torch.randint(0, V, (N,), generator=g, device=DEV)


@pytest.mark.parametrize("N,V,H,dtype,wide", [(1, 1, 1, FP32, True), (1, 50, 2560, BF16, False), (7, 9, 33, BF16, True),
                                              (300, 1000, 96, FP16, False), (513, 4097, 130, FP32, True)])
def test_embed(N, V, H, dtype, wide):
    g = gen(N + V)
    table, ids = randn(g, V, H, dtype=dtype), token_ids(g, N, V, "all")
    new = Guarded()
    out = new((N, H), dtype)
    ftmoe.ftmoe_embed(table, V, H, ids if wide else ids.int(), N, 1.7, out)
    torch.cuda.synchronize()
    new.check()
    ref = table[ids].double() * float(np.float32(1.7))
    within(out, ref, (UNIT[dtype] + 2 * EPS) * ref.abs() + TINY[dtype])
    ftmoe.ftmoe_embed(table, V, H, ids if wide else ids.int(), N, 1.0, out)
    assert torch.equal(out, table[ids])


def test_embed_ids_out_of_range():
    table, out = randn(gen(0), 5, 16, dtype=BF16), torch.ones(4, 16, dtype=BF16, device=DEV)
    ids = torch.tensor([4, 5, -1, 1 << 33], device=DEV)
    ftmoe.ftmoe_embed(table, 5, 16, ids, 4, 1.0, out)
    assert ftmoe.ftmoe_ops_status() == -10
    assert torch.equal(out[0], table[4]) and not out[1:].any()


def embed_backward(dout, ids, V, scale, table, padding=-1, accumulate=False):
    N, H = dout.shape
    new = Guarded()
    ws = new((ftmoe.ftmoe_embed_workspace(N, H),), torch.uint8)
    dtable = new(table.shape, table.dtype)
    dtable.copy_(table)
    ftmoe.ftmoe_embed_backward(dout, ids, N, V, H, scale, padding, dtable, accumulate, ws)
    torch.cuda.synchronize()
    new.check()
    return dtable


@pytest.mark.parametrize("N,V,H,dtype,tdtype,kind,wide", [
    (0, 3, 8, BF16, BF16, "all", True), (1, 1, 1, FP32, FP32, "one", False), (1, 5000, 64, BF16, BF16, "all", True),
    (31, 7, 33, BF16, FP32, "few", True), (32, 7, 40, FP16, FP16, "one", False), (33, 2, 40, FP16, FP32, "one", True),
    (64, 600, 1001, BF16, BF16, "few", False), (65, 64, 256, FP32, FP32, "all", True),
    (1000, 100000, 24, BF16, BF16, "all", True), (3000, 9, 288, BF16, FP32, "few", False),
    (5000, 1 << 20, 4, FP32, FP32, "all", False), (2048, 3, 12, BF16, BF16, "one", True)])
def test_embed_backward(N, V, H, dtype, tdtype, kind, wide):
    g = gen(N + 3 * V)
    dout, ids = randn(g, N, H, dtype=dtype), token_ids(g, N, V, kind)
    stale = torch.full((V, H), 7.0, dtype=tdtype, device=DEV)
    got = embed_backward(dout, ids if wide else ids.int(), V, 0.5, stale)
    ref = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, dout.double()) * 0.5
    size = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, dout.double().abs()) * 0.5
    n = torch.bincount(ids, minlength=V)[:, None].double()
    within(got, ref, UNIT[tdtype] * 1.01 * ref.abs() + 2 * (n + 2) * EPS * size + TINY[tdtype] * (n > 0))
    again = embed_backward(dout, ids if wide else ids.int(), V, 0.5, stale)
    assert torch.equal(got, again)  # no order that changes


def test_embed_backward_adds_onto_the_table():
    g = gen(4)
    N, V, H = 100, 50, 36
    dout, ids, start = randn(g, N, H, dtype=BF16), token_ids(g, N, V, "few"), randn(g, V, H)
    got = embed_backward(dout, ids, V, 2.0, start, accumulate=True)
    add = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, dout.double()) * 2
    size = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, dout.double().abs()) * 2
    within(got, start.double() + add, 2 * 102 * EPS * size + 2 * EPS * (start.double() + add).abs())
    free = torch.bincount(ids, minlength=V) == 0
    assert torch.equal(got[free], start[free])


@pytest.mark.parametrize("H,dtype", [(64, BF16), (36, torch.float32), (33, torch.float16)])
@pytest.mark.parametrize("N,V,kind", [(1, 5, "all"), (700, 90, "all"), (3000, 40, "few"), (5000, 7000, "all")])
def test_embed_backward_adds_runs_of_every_length(N, V, kind, H, dtype):
    """Vector and single additions, rows of one token, of a chunk's and of many chunks'."""
    g = gen(N + H)
    dout, ids, start = randn(g, N, H, dtype=dtype), token_ids(g, N, V, kind), randn(g, V, H)
    got = embed_backward(dout, ids, V, 0.7, start, accumulate=True)
    scale = float(torch.tensor(0.7))  # as fp32 holds it
    add = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, dout.double()) * scale
    size = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, dout.double().abs()) * scale
    n = torch.bincount(ids, minlength=V)[:, None].double()
    within(got, start.double() + add, 2 * (n + 2) * EPS * size + 2 * EPS * (start.double() + add).abs())
    assert torch.equal(got[n[:, 0] == 0], start[n[:, 0] == 0])
    assert torch.equal(got, embed_backward(dout, ids, V, 0.7, start, accumulate=True))


@pytest.mark.parametrize("V", [511, 512, 1000, 1023, 1024, 300000, 1 << 20])
def test_embed_backward_of_many_tokens(V):
    """Wider digits: one pass up to 1023 rows, two up to 2^20 - 1, three beyond."""
    N, H = 66001, 8
    g = gen(V)
    dout, ids = randn(g, N, H, dtype=BF16), token_ids(g, N, V, "all")
    got = embed_backward(dout, ids.int(), V, 1.0, torch.full((V, H), 7.0, device=DEV), padding=V - 1)
    use = ids != V - 1
    ref = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[use], dout[use].double())
    size = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[use], dout[use].double().abs())
    n = torch.bincount(ids[use], minlength=V)[:, None].double()
    within(got, ref, 2 * (n + 2) * EPS * size)


def test_embed_backward_padding_and_bad_ids():
    g = gen(5)
    N, V, H = 200, 20, 16
    dout, ids = randn(g, N, H), token_ids(g, N, V, "all")
    ids[::3] = 6
    stale = torch.full((V, H), 7.0, device=DEV)
    got = embed_backward(dout, ids, V, 1.0, stale, padding=6)
    use = ids != 6
    ref = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[use], dout[use].double())
    size = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[use], dout[use].double().abs())
    within(got, ref, 2 * (N + 2) * EPS * size)
    assert not got[6].any() and ftmoe.ftmoe_ops_status() == 0
    odd = ids.clone()
    odd[1], odd[2] = V, -3
    use[1] = use[2] = False
    got = embed_backward(dout, odd, V, 1.0, stale, padding=6)
    ref = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids[use], dout[use].double())
    within(got, ref, 2 * (N + 2) * EPS * size)
    assert ftmoe.ftmoe_ops_status() == -10


def test_embed_and_its_gradient_are_adjoint():
    g = gen(6)
    N, V, H = 90, 40, 52
    table, d, ids = randn(g, V, H), randn(g, N, H), token_ids(g, N, V, "few")
    out = torch.empty(N, H, device=DEV)
    ftmoe.ftmoe_embed(table, V, H, ids, N, 3.0, out)
    grad = embed_backward(d, ids, V, 3.0, table)
    size = float((out.double() * d.double()).abs().sum())
    assert abs(float((out.double() * d.double()).sum()) - float((grad.double() * table.double()).sum())) <= \
        2 * (N + 4) * EPS * size


# ----------------------------------------------------------------- policy loss

def policy_inputs(seed, N, V, dtype, masked=0.3, ld=None, at=0):
    """Rows `ld` apart, the first `at` values into its buffer."""
    g = gen(seed)
    ld = V if ld is None else ld
    raw = randn(g, at + N * ld, dtype=dtype, std=2.5)
    logits = raw[at:].view(N, ld)[:, :V]
    y = torch.randint(0, V, (N,), generator=g, device=DEV)
    z = logits.double()
    lp = torch.log_softmax(z, 1).gather(1, y[:, None])[:, 0].float()
    keep = (torch.rand(N, generator=g, device=DEV) >= masked).float()
    return dict(logits=logits, targets=y, old_logp=lp + 0.3 * randn(g, N), ref_logp=lp + 0.3 * randn(g, N),
                advantage=randn(g, N), weight=keep / keep.sum().clamp(min=1))


def policy(i, grad=True, logp=True, in_place=False, ld_d=None, **kw):
    logits = i["logits"]
    N, V = logits.shape
    new = Guarded()
    loss, row, lp = new((1,), FP32), new((N,), FP32), new((N,), FP32) if logp else None
    d = None
    if in_place:
        d = logits
    elif grad:
        d = new((N, ld_d or V), logits.dtype, 7.0)
    a = ftmoe.policy_args(i["logits"], i["targets"], i["old_logp"], i["ref_logp"], i["advantage"], i["weight"], loss,
                          row, lp, d[:, :V] if d is not None else None, **kw)
    ftmoe.ftmoe_policy_loss(a)
    torch.cuda.synchronize()
    new.check()
    if ld_d:
        assert bool((d[:, V:] == 7.0).all())
        d = d[:, :V]
    return loss, row, lp, d


def policy_check(i, outs, dtype, temperature=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.0, grad_scale=1.0):
    loss, row, lp, d = outs
    f = lambda v: float(np.float32(v))
    temperature, lo, hi, b, gs = f(temperature), f(clip_low), f(clip_high), f(kl_coef), f(grad_scale)
    z = i["logits"].double() / temperature
    N, V = z.shape
    y, use = i["targets"].long()[:, None], None
    w = i["weight"].double() if i["weight"] is not None else torch.full((N,), 1 / N, dtype=torch.float64, device=DEV)
    use = w != 0
    ref_lp = z.gather(1, y)[:, 0] - torch.logsumexp(z, 1)
    size = torch.where(torch.isfinite(z), z, 0.0).abs().amax(1)
    # the exponential and its argument, the sum's additions per thread and across threads, the logarithm
    dl = 2 * EPS * (V / 512 + 64 + 6 * size)
    if lp is not None:
        within(lp, torch.where(use, ref_lp, 0.0), dl)
    A, x = i["advantage"].double(), ref_lp - i["old_logp"].double()
    r = torch.exp(x)
    dr = r * (dl + 2 * EPS * (4 + x.abs()))
    cl = torch.clamp(r, 1 - lo, 1 + hi)
    clipped = r * A > cl * A
    ref_row, drow = -torch.where(clipped, cl * A, r * A), A.abs() * (dr + 4 * EPS * (r + cl))
    c, dc = torch.where(clipped, 0.0, -r * A), A.abs() * (dr + 4 * EPS * r)
    if i["ref_logp"] is not None and b:
        t = i["ref_logp"].double() - ref_lp
        e = torch.exp(t)
        de = e * (dl + 2 * EPS * (4 + t.abs()))
        ref_row, drow = ref_row + b * (e - t - 1), drow + b * (de + dl + 4 * EPS * (e + t.abs() + 1))
        c, dc = c + b * (1 - e), dc + b * (de + 4 * EPS * (e + 1))
    # a ratio within its error of a corner may fall on either side: the row is the same there, its slope either's
    corner = torch.minimum((r - (1 - lo)).abs(), (r - (1 + hi)).abs()) <= 2 * dr
    assert int(corner.sum()) <= 1 + N // 100
    dc = dc + torch.where(corner, r * A.abs(), 0.0)
    ref_row, drow = torch.where(use, ref_row, 0.0), torch.where(use, drow, 0.0)
    within(row, ref_row, drow)
    within(loss[0], (w * ref_row).sum(), (w.abs() * drow).sum() + 4 * EPS * (w * ref_row).abs().sum())
    if d is None:
        return
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    hot = torch.zeros_like(p).scatter_(1, y, 1.0)
    k = gs * w / temperature
    ref = torch.where(use[:, None], (k * c)[:, None] * (hot - p), 0.0)
    err = (k.abs() * (dc + 6 * EPS * c.abs()))[:, None] * (hot + p) + (k * c).abs()[:, None] * p * (2 * dl[:, None])
    within(d, ref, UNIT[dtype] * 1.01 * ref.abs() + torch.where(use[:, None], err, 0.0) + TINY[dtype])


@pytest.mark.parametrize("N,V,dtype,ld,at", [
    (1, 1, FP32, None, 0), (3, 2, BF16, None, 0), (5, 7, FP16, None, 1), (40, 1000, BF16, None, 0),
    (17, 333, BF16, 340, 3), (9, 4097, FP32, None, 2), (2, 50001, BF16, None, 0), (6, 20011, FP16, 20012, 5),
    (1, 131072, BF16, None, 0), (700, 65, FP32, None, 0), (2, 200003, FP32, None, 1), (2, 500003, FP32, None, 1),
    (2100, 2051, BF16, None, 1), (900, 8200, FP32, None, 0), (600, 16001, FP16, 16005, 2)])
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_policy_loss(N, V, dtype, ld, at, masked):
    i = policy_inputs(N + V, N, V, dtype, masked, ld, at)
    kw = dict(temperature=0.8, clip_low=0.2, clip_high=0.3, kl_coef=0.05, grad_scale=64.0)
    policy_check(i, policy(i, **kw), dtype, **kw)
    kw = dict(temperature=1.0, clip_low=0.1, clip_high=0.1)
    outs = policy(i, grad=False, **kw)
    policy_check(i, outs, dtype, **kw)
    with_grad = policy(i, **kw)
    for a, b in zip(outs[:3], with_grad[:3]):  # the gradient changes no bit of the forward
        assert torch.equal(a, b)
    odd = policy(i, ld_d=V + 3, **kw)  # gradient rows of another alignment
    assert torch.equal(odd[3], with_grad[3])
    inp = policy(i, in_place=True, **kw)  # last: it overwrites the logits
    assert torch.equal(inp[3], with_grad[3]) and torch.equal(inp[0], outs[0])


def test_policy_loss_optional_parts():
    N, V = 21, 130
    i = policy_inputs(9, N, V, BF16)
    i["targets"] = i["targets"].int()
    i["weight"] = i["ref_logp"] = None
    policy_check(i, policy(i, kl_coef=0.1), BF16)
    assert policy(i, logp=False)[2] is None
    empty = {k: v[:0] for k, v in policy_inputs(9, 4, 8, BF16).items()}
    assert float(policy(empty)[0]) == 0.0


def test_policy_loss_masked_rows_are_not_read():
    N, V = 12, 77
    i = policy_inputs(10, N, V, FP32, masked=0.0)
    i["weight"][::2] = 0.0
    clean = policy(i, kl_coef=0.1)
    for name in ("logits", "old_logp", "ref_logp", "advantage"):
        i[name][::2] = float("nan")
    dirty = policy(i, kl_coef=0.1)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    assert not dirty[3][::2].any() and not dirty[1][::2].any()
    i["weight"].zero_()
    loss, row, lp, d = policy(i, kl_coef=0.1)
    assert float(loss) == 0.0 and not row.any() and not lp.any() and not d.any()


@pytest.mark.parametrize("V", [50, 70000])
def test_policy_loss_of_infinite_and_nan_logits(V):
    N = 4
    i = policy_inputs(11, N, V, FP32, masked=0.0)
    i["logits"][0, ::2] = -float("inf")  # a vocabulary mask
    i["targets"][0] = 1
    lp = torch.log_softmax(i["logits"][0].double(), 0)[1]
    i["old_logp"][0] = i["ref_logp"][0] = float(lp)
    i["logits"][1] = -float("inf")
    i["logits"][1, 3] = -1e30  # the only value left, very low
    i["targets"][1] = 3
    i["old_logp"][1] = i["ref_logp"][1] = 0.0
    loss, row, lp, d = policy(i, kl_coef=0.1)
    policy_check({k: v[:1] for k, v in i.items()}, (row[:1].double() * i["weight"][:1], row[:1], lp[:1], d[:1]), FP32,
                 kl_coef=0.1)
    assert float(lp[1]) == 0.0 and not d[0, ::2].any()
    assert float(d[1].abs().max()) <= 1e-6  # softmax is the target alone
    i["logits"][2, 5] = float("nan")
    i["logits"][3] = -float("inf")
    loss, row, lp, d = policy(i, kl_coef=0.1)
    assert bool(torch.isnan(loss)) and bool(torch.isnan(row[2:]).all()) and bool(torch.isnan(d[2:]).all())
    assert bool(torch.isfinite(d[:2]).all())


def test_policy_loss_bad_targets():
    i = policy_inputs(12, 6, 30, BF16, masked=0.0)
    i["targets"][1], i["targets"][4] = 30, -1
    loss, row, lp, d = policy(i, kl_coef=0.1)
    assert ftmoe.ftmoe_ops_status() == -10
    assert not d[[1, 4]].any() and not row[[1, 4]].any() and bool(d[[0, 2, 3, 5]].any(1).all())


def test_policy_gradient_against_differences():
    """A central difference of the kernel's own loss along a random direction."""
    N, V, h = 16, 50, 2.0 ** -7
    i = policy_inputs(13, N, V, FP32, masked=0.25)
    # ratios away from the clip's corners, so that the loss is smooth within the step
    for n in range(N):
        i["old_logp"][n] = float(torch.log_softmax(i["logits"][n].double(), 0)[i["targets"][n]]) - [0.0, 0.6, -0.6, 0.05][n % 4]
    kw = dict(kl_coef=0.2, clip_low=0.2, clip_high=0.2)
    direction = randn(gen(14), N, V)
    direction /= direction.abs().amax(1, keepdim=True)
    d = policy(i, **kw)[3].double()
    start = i["logits"].clone()
    vals = []
    for s in (h, -h):
        i["logits"] = start + s * direction
        vals.append(policy(i, grad=False, **kw)[1].double())
    w = i["weight"].double()
    slope = (w * (vals[0] - vals[1]) / (2 * h)).sum()
    # third derivatives of a row are below 8 (1 + |A| r + b e^d) for a direction of unit maximum; fp32 row errors over 2h
    size = (w * (1 + i["advantage"].abs().double() * 2 + 1)).sum()
    assert abs(float(slope - (d * direction.double()).sum())) <= float(size) * (8 * h * h / 6 * 8 + 2 * EPS * 200 / h)


# ----------------------------------------------------------------- AdamW

def e4m3_table():
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


TABLE = e4m3_table()


def e4m3_codes(x):
    """Codes of fp32 values, to the nearest value of the format, ties to the even code."""
    a = np.abs(x).astype(np.float64)
    hi = np.searchsorted(TABLE, a).clip(0, 126)
    lo = (hi - 1).clip(0)
    up, down = TABLE[hi] - a, a - TABLE[lo]
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    c = np.where(a >= 448, 126, c)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def adam_case(seed, sizes, dtype, gdtype, master, bits, offset=0):
    """Tensors of these sizes, `offset` values into buffers of their own."""
    g, out = gen(seed), []
    for k, n in enumerate(sizes):
        new = Guarded()

        def take(dt, std, n=n, positive=False):
            t = new((n + offset,), dt)[offset:]
            v = randn(g, n, std=std)
            t.copy_((v.abs() if positive else v).to(dt))
            return t
        t = dict(p=take(dtype, 1.0), g=take(gdtype, 0.1), weight_decay=[0.0, 0.1][k % 2], guard=new)
        if master:
            t["master"] = new((n + offset,), FP32)[offset:]
            t["master"].copy_(t["p"].float() + randn(g, n, std=1e-3))
        if bits == 32:
            t["m"], t["v"] = take(FP32, 0.01), take(FP32, 1e-4, positive=True)
        else:
            blocks = -(-n // 256)
            for name in ("m", "v"):
                codes = torch.randint(0, 127, (n,), generator=g, device=DEV)
                if name == "m":
                    codes = codes | (torch.randint(0, 2, (n,), generator=g, device=DEV) << 7)
                t[name] = new((n + offset,), torch.uint8)[offset:]
                t[name].copy_(codes.to(torch.uint8))
                t[name + "_scale"] = new((blocks,), FP32)
                t[name + "_scale"].copy_(torch.rand(blocks, generator=g, device=DEV) * 1e-4 + 1e-6)
        out.append(t)
    return out


def decoded(codes, scale):
    v = np.concatenate([TABLE, [np.nan], -TABLE, [np.nan]])[codes].astype(np.float32)
    return v * np.repeat(scale, 256)[:len(codes)]


def adam_check(t, before, hp, gs):
    f = np.float32
    host = lambda v: v.float().cpu().numpy() if v.dtype != torch.uint8 else v.cpu().numpy()
    eight = t["m"].dtype == torch.uint8
    g = host(before["g"]).astype(np.float32) * f(gs)
    if eight:
        m, u = decoded(host(before["m"]), host(before["m_scale"])), decoded(host(before["v"]), host(before["v_scale"]))
        v = u * u
    else:
        m, v = host(before["m"]), host(before["v"])
    # 64 bits from the same fp32 inputs
    m64 = hp["beta1"] * m.astype(np.float64) + (1 - hp["beta1"]) * g.astype(np.float64)
    v64 = hp["beta2"] * v.astype(np.float64) + (1 - hp["beta2"]) * g.astype(np.float64) ** 2
    c1, c2 = 1 - hp["beta1"] ** hp["step"], 1 - hp["beta2"] ** hp["step"]
    update = hp["lr"] / c1 * m64 / (np.sqrt(v64 / c2) + hp["eps"])
    old = host(before["master"] if "master" in t else before["p"]).astype(np.float64)
    p64 = old * (1 - hp["lr"] * t["weight_decay"]) - update
    merr = 8 * EPS * (np.abs(hp["beta1"] * m.astype(np.float64)) + np.abs(g) * (1 - hp["beta1"]))
    # m's error and twelve roundings of the quotient and its parts
    perr = 4 * EPS * (np.abs(old) + np.abs(p64)) + 24 * EPS * np.abs(update) + \
        hp["lr"] / c1 * merr / (np.sqrt(v64 / c2) + hp["eps"]) + 2.0 ** -126
    if "master" in t:
        within(t["master"], p64, perr)
        assert torch.equal(t["p"], t["master"].to(t["p"].dtype))
    else:
        u = UNIT[t["p"].dtype]
        within(t["p"], p64, u * 1.01 * np.abs(p64) + perr + TINY[t["p"].dtype])
    if not eight:
        within(t["m"], m64, merr + 2.0 ** -126)
        within(t["v"], v64, 8 * EPS * v64 + 2.0 ** -126)
        return
    # the codes are those of the formula in fp32, bit for bit
    m32 = m * f(hp["beta1"]) + g * f(1 - hp["beta1"])
    v32 = v * f(hp["beta2"]) + g * g * f(1 - hp["beta2"])
    for name, x in (("m", m32), ("v", np.sqrt(v32))):
        n = len(x)
        pad = np.zeros(-(-n // 256) * 256, np.float32)
        pad[:n] = x
        top = np.abs(pad.reshape(-1, 256)).max(1)
        with np.errstate(divide="ignore"):
            r = np.where(top < f(1e-30), f(0), f(448) * (f(1) / top)).astype(np.float32)
        codes = e4m3_codes(x * np.repeat(r, 256)[:n])
        if name == "v":
            codes = np.where((codes == 0) & (x > 0) & (np.repeat(top, 256)[:n] >= f(1e-30)), 1, codes)
        scale = np.where(top < f(1e-30), f(0), top * (f(1) / f(448))).astype(np.float32)
        assert np.array_equal(host(t[name + "_scale"]), scale), name
        assert np.array_equal(host(t[name]), codes), name


SIZES = [1, 255, 256, 257, 2048, 2049, 5000, 7, 4096]


@pytest.mark.parametrize("dtype,gdtype,master", [(BF16, BF16, True), (BF16, FP32, False), (FP16, FP16, False),
                                                 (FP16, FP32, True), (FP32, FP32, False)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("offset", [0, 1])
def test_adamw(dtype, gdtype, master, bits, offset):
    ts = adam_case(17 + bits + offset, SIZES, dtype, gdtype, master, bits, offset)
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=3)
    scale = torch.full((1,), 0.75, device=DEV)
    lst = ftmoe.adamw_list(ts)
    for step in range(2):
        before = [{k: v.clone() for k, v in t.items() if torch.is_tensor(v)} for t in ts]
        hp["step"] += 1
        ftmoe.ftmoe_adamw(lst, grad_scale=scale, **hp)
        torch.cuda.synchronize()
        for t, b in zip(ts, before):
            t["guard"].check()
            assert torch.equal(t["g"], b["g"])
            adam_check(t, b, hp, 0.75)


def test_adamw_mixed_list_and_many_tensors():
    """Kinds in one list, and more tensors than one launch carries."""
    ts = []
    for k, (dt, gd, ms, bits) in enumerate([(BF16, BF16, True, 32), (FP32, FP32, False, 8), (FP16, FP32, False, 32)]):
        ts += adam_case(40 + k, [3, 300], dt, gd, ms, bits)
    ts += adam_case(50, [5] * 900, BF16, BF16, False, 32)
    ts.insert(3, dict(p=torch.empty(0, device=DEV), g=torch.empty(0, device=DEV), m=torch.empty(0, device=DEV),
                      v=torch.empty(0, device=DEV)))
    before = [{k: v.clone() for k, v in t.items() if torch.is_tensor(v)} for t in ts]
    hp = dict(lr=1e-3, beta1=0.0, beta2=0.999, eps=1e-6, step=1)
    ftmoe.ftmoe_adamw(ftmoe.adamw_list(ts), **hp)
    torch.cuda.synchronize()
    for t, b in zip(ts, before):
        if t["p"].numel():
            t["guard"].check()
            adam_check(t, b, hp, 1.0)


def test_adamw_8bit_from_zero_state_and_zero_gradients():
    ts = adam_case(60, [600], FP32, FP32, False, 8)
    t = ts[0]
    for n in ("m", "v", "m_scale", "v_scale"):
        t[n].zero_()
    t["g"][256:512] = 0.0  # a block that stays zero
    t["g"][0], t["g"][1] = 1e4, 1e-3  # a root far below its block's largest keeps a code
    before = {k: v.clone() for k, v in t.items() if torch.is_tensor(v)}
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)
    ftmoe.ftmoe_adamw(ftmoe.adamw_list(ts), **hp)
    torch.cuda.synchronize()
    adam_check(t, before, hp, 1.0)
    assert not t["m"][256:512].any() and float(t["v_scale"][1]) == 0.0 and int(t["v"][1]) == 1
    assert torch.equal(t["p"][256:512], before["p"][256:512] * float(np.float32(1.0)))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_adamw_skips_an_overflowed_step(value):
    ts = adam_case(61, [700], BF16, BF16, True, 32) + adam_case(62, [700], BF16, BF16, False, 8)
    before = [{k: v.clone() for k, v in t.items() if torch.is_tensor(v)} for t in ts]
    ftmoe.ftmoe_adamw(ftmoe.adamw_list(ts), lr=1.0, grad_scale=torch.full((1,), value, device=DEV))
    torch.cuda.synchronize()
    for t, b in zip(ts, before):
        assert all(torch.equal(t[k], b[k]) for k in b)


# ----------------------------------------------------------------- streams and graphs

def test_other_streams_and_graph_replay():
    """A side stream gives the same bits, and a captured step replays on new inputs."""
    T, k, E, H, V = 600, 8, 32, 64, 300
    g = gen(70)
    idx, x, w = choose(g, T, k, E, 0.1), randn(g, T, H, dtype=BF16), torch.rand(T, k, generator=g, device=DEV)
    ids, P = token_ids(g, T, V, "few"), T * k
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)
    off, perm, inv = i32(E + 1), i32(P), i32(P)
    xs, out, dys = (torch.zeros(n, H, dtype=BF16, device=DEV) for n in (P, T, P))
    dw, table = torch.empty(T, k, device=DEV), torch.empty(V, H, dtype=BF16, device=DEV)
    ws = torch.empty(ftmoe.ftmoe_embed_workspace(T, H), dtype=torch.uint8, device=DEV)
    i = policy_inputs(71, 40, 500, BF16)
    loss, row, lp, dl = (torch.empty(n, device=DEV) for n in (1, 40, 40, 1))
    dl = torch.empty_like(i["logits"])
    a = ftmoe.policy_args(*(i[n] for n in ("logits", "targets", "old_logp", "ref_logp", "advantage", "weight")), loss,
                          row, lp, dl, kl_coef=0.1)

    def step(stream=None):
        ftmoe.ftmoe_dispatch(x, T, H, idx, k, E, off, perm, inv, xs, stream=stream)
        ftmoe.ftmoe_combine(xs, T, H, k, inv, w, out, stream=stream)
        ftmoe.ftmoe_combine_backward(out, xs, T, H, k, inv, w, dys, dw, stream=stream)
        ftmoe.ftmoe_embed_backward(out, ids, T, V, H, 1.0, -1, table, False, ws, stream=stream)
        ftmoe.ftmoe_policy_loss(a, stream=stream)
    results = (off, perm, inv, xs, out, dys, dw, table, loss, row, lp, dl)
    step()
    torch.cuda.synchronize()
    want = [r.clone() for r in results]
    for r in results:
        r.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(r, v) for r, v in zip(results, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2, idx2 = randn(g, T, H, dtype=BF16), choose(g, T, k, E, 0.1)
    x.copy_(x2)
    idx.copy_(idx2)
    for r in results:
        r.zero_()
    graph.replay()
    torch.cuda.synchronize()
    replayed = [r.clone() for r in results]
    for r in results:
        r.zero_()
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(r, v) for r, v in zip(results, replayed))


def test_strided_tensors_are_refused():
    x = torch.zeros(8, 32, dtype=BF16, device=DEV)[:, ::2]
    i = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    o = torch.zeros(64, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        ftmoe.ftmoe_dispatch(x, 8, 16, i, 2, 4, o, o, o, x)
    with pytest.raises(TypeError):
        ftmoe.ftmoe_combine(x.contiguous().double(), 8, 16, 2, o, None, x.contiguous())
    z = torch.zeros(4, 10, device=DEV)
    with pytest.raises(ValueError):
        ftmoe.policy_args(z.t(), o, o, o, o, o, o, o)


# ----------------------------------------------------------------- offsets past 32 bits

def test_lookup_and_gradient_in_a_table_past_32_bits():
    V, H, N = 600_000, 4096, 64  # 2.46e9 values
    g = gen(80)
    table = torch.empty(V, H, dtype=BF16, device=DEV)
    ids = torch.cat([torch.arange(V - 40, V, device=DEV), torch.randint(0, V, (N - 40,), generator=g, device=DEV)])
    table[ids] = randn(g, N, H, dtype=BF16)
    out = torch.empty(N, H, dtype=BF16, device=DEV)
    ftmoe.ftmoe_embed(table, V, H, ids, N, 1.0, out)
    assert torch.equal(out, table[ids])
    table.fill_(7.0)
    ws = torch.empty(ftmoe.ftmoe_embed_workspace(N, H), dtype=torch.uint8, device=DEV)
    ids[40:] = V - 1  # a run past its chunk
    ftmoe.ftmoe_embed_backward(out, ids, N, V, H, 1.0, -1, table, False, ws)
    assert torch.equal(table[V - 40:V - 1], out[:39])
    last = out[39:].double().sum(0)
    within(table[V - 1], last, UNIT[BF16] * 1.01 * last.abs() + 2 * 27 * EPS * out[39:].double().abs().sum(0))
    assert not any(bool(table[a:a + 100_000].any()) for a in range(0, V - 100_000, 100_000))


def test_dispatch_and_combine_past_32_bits():
    T, k, E, H = 70_000, 8, 16, 4096  # 2.29e9 values in sorted order
    g = gen(81)
    idx = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    x = randn(g, T, H, dtype=BF16)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)
    off, perm, inv, xs = i32(E + 1), i32(T * k), i32(T * k), torch.empty(T * k, H, dtype=BF16, device=DEV)
    ftmoe.ftmoe_dispatch(x, T, H, idx, k, E, off, perm, inv, xs)
    ordered, order = torch.sort(idx.view(-1), stable=True)
    assert torch.equal(perm, order.int())
    for a in range(0, T * k, 80_000):
        assert torch.equal(xs[a:a + 80_000], x[order[a:a + 80_000] // k])
    out = torch.empty(T, H, dtype=BF16, device=DEV)
    ftmoe.ftmoe_combine(xs, T, H, k, inv, torch.full((T, k), 0.125, device=DEV), out)
    assert torch.equal(out, x)  # eight times an eighth of the row, exactly
    dw = torch.empty(T, k, device=DEV)
    ftmoe.ftmoe_combine_backward(x, xs, T, H, k, inv, torch.full((T, k), 2.0, device=DEV), xs, dw)
    for a in range(0, T * k, 80_000):
        assert torch.equal(xs[a:a + 80_000], 2 * x[order[a:a + 80_000] // k])
    square = x[-100:].double().square().sum(1, keepdim=True)
    within(dw[-100:], square.expand(-1, k), 2 * (H + 2) * EPS * square)


def test_policy_loss_past_32_bits():
    N, V = 17_000, 131_072  # 2.23e9 logits
    g = gen(82)
    logits = torch.empty(N, V, dtype=BF16, device=DEV)
    logits.fill_(-3.0)
    few = policy_inputs(83, 50, V, BF16, masked=0.0)
    logits[N - 50:] = few["logits"]
    i = dict(logits=logits, weight=torch.zeros(N, device=DEV), targets=torch.zeros(N, dtype=torch.int64, device=DEV))
    for n in ("old_logp", "ref_logp", "advantage", "targets", "weight"):
        i.setdefault(n, torch.zeros(N, device=DEV))
        i[n][N - 50:] = few[n]
    want = policy(few, kl_coef=0.1)
    got = policy(i, in_place=True, kl_coef=0.1)
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[N - 50:], b)
    assert not got[1][:N - 50].any() and not logits[:N - 50:997].any()


def test_adamw_past_32_bits():
    n, tail = (1 << 31) + 1000, 2048 * 3  # the tail's blocks start on a block's boundary
    g = gen(84)
    start = (n - tail) // 256 * 256
    big = dict(p=torch.zeros(n, dtype=BF16, device=DEV), g=torch.zeros(n, dtype=BF16, device=DEV),
               m=torch.zeros(n, dtype=torch.uint8, device=DEV), v=torch.zeros(n, dtype=torch.uint8, device=DEV),
               m_scale=torch.zeros(-(-n // 256), device=DEV), v_scale=torch.zeros(-(-n // 256), device=DEV),
               weight_decay=0.1)
    big["p"][start:] = randn(g, n - start, dtype=BF16)
    big["g"][start:] = randn(g, n - start, dtype=BF16)
    small = {k: v[start // 256 if "scale" in k else start:].clone() if torch.is_tensor(v) else v for k, v in big.items()}
    for t in (big, small):
        ftmoe.ftmoe_adamw(ftmoe.adamw_list([t]), lr=1e-2, step=1)
    for k, v in small.items():
        if torch.is_tensor(v):
            assert torch.equal(big[k][start // 256 if "scale" in k else start:], v), k
    assert not big["p"][:start:99_991].any() and not big["v"][:start:99_991].any()


@pytest.mark.parametrize("N,V,dtype", [(1300, 4500, BF16), (1217, 6001, FP32), (1250, 12007, FP16)])
def test_policy_loss_rows_of_two_warps(N, V, dtype):
    """Many rows of 8 to 24 KB: two warps a row, several rows a CTA in turn."""
    i = policy_inputs(90 + V, N, V, dtype, 0.3)
    kw = dict(temperature=1.1, kl_coef=0.05)
    policy_check(i, policy(i, **kw), dtype, **kw)
    a, b = policy(i, grad=False, **kw), policy(i, **kw)
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)
