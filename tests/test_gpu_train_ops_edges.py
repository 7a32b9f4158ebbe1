"""Edges of the training operators that the sizes and inputs elsewhere do not
reach.  Bounds are those that test_gpu_train_ops derives, restated where a
test's quantity differs."""

import threading
import time

import numpy as np
import pytest
import torch

from nvfp4_mixture_experts_counting_gb300 import ftmoe

import test_gpu_train_ops as base
from test_gpu_train_ops import (BF16, DEV, EPS, FP16, FP32, TINY, UNIT, gen, policy, policy_check, policy_inputs,
                                randn, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from nvfp4_mixture_experts_counting_gb300 import build
    build.build()
    ftmoe.ftmoe_ops_status()
    yield
    assert ftmoe.ftmoe_ops_status() == 0  # every test that marks the word reads it


# ----------------------------------------------------------------- policy loss: one slope a row

# a warp a row, two warps, four, clusters of CTAs, and rows that are read twice
ROWS = [(700, 65, FP32), (1300, 2049, BF16), (1300, 4500, BF16), (1217, 6001, FP32), (300, 16001, FP16),
        (64, 131072, BF16), (200, 50001, FP32), (6, 500003, FP32), (6, 1000003, BF16)]


@pytest.mark.parametrize("N,V,dtype", ROWS)
def test_a_row_at_a_clip_bound_has_one_slope(N, V, dtype):
    """clip 0 and old_logp the call's own: every ratio is within rounding of both bounds, so either side may
    be taken, but by all of a row: it is zeros, or -A r (onehot - softmax) w."""
    i = policy_inputs(N + V, N, V, dtype, masked=0.0)
    i["ref_logp"] = None
    i["old_logp"] = policy(i, grad=False)[2]
    d = policy(i, clip_low=0.0, clip_high=0.0)[3].double()
    z, y = i["logits"].double(), i["targets"][:, None]
    p = torch.softmax(z, 1)
    hot = torch.zeros_like(p).scatter_(1, y, 1.0)
    logp = (z.gather(1, y)[:, 0] - torch.logsumexp(z, 1))
    dl = 2 * EPS * (V / 512 + 64 + 6 * z.abs().amax(1))
    x = logp - i["old_logp"].double()
    r, k, A = torch.exp(x), i["weight"].double(), i["advantage"].double()
    dr = r * (dl + 2 * EPS * (4 + x.abs()))
    ref = (-k * A * r)[:, None] * (hot - p)
    err = (k * A.abs() * (dr + 10 * EPS * r))[:, None] * (hot + p) + (k * A * r).abs()[:, None] * p * (2 * dl[:, None])
    slope = ((d - ref).abs() <= UNIT[dtype] * 1.01 * ref.abs() + err + TINY[dtype]).all(1)
    zeros = (d == 0).all(1)
    assert bool((slope | zeros).all()), int((~(slope | zeros)).sum())


@pytest.mark.parametrize("N,V,dtype", ROWS)
def test_equal_logits_have_equal_gradients(N, V, dtype):
    """A row of one value: its gradient is one value off the target, to the last bit."""
    i = policy_inputs(N + V, N, V, dtype, masked=0.0)
    i["logits"] = i["logits"][:, :1].expand(N, V).contiguous()
    lp = -float(np.log(V))
    i["old_logp"] = lp + 0.1 * torch.sin(torch.arange(N, device=DEV).float())
    i["ref_logp"] = lp + 0.1 * torch.cos(torch.arange(N, device=DEV).float())
    d = policy(i, kl_coef=0.3, clip_low=0.5, clip_high=0.5, grad_scale=4096.0)[3]
    other = (i["targets"] == 0).long()[:, None]
    value = d.gather(1, other)  # of a column that is not the target's
    off = torch.ones(N, V, dtype=torch.bool, device=DEV).scatter_(1, i["targets"][:, None], False)
    assert bool(((d == value) | ~off).all())


# ----------------------------------------------------------------- policy loss: next to the reference

@pytest.mark.parametrize("N,V,dtype", [(1000, 3000, FP32), (300, 16001, BF16), (64, 131072, BF16), (4, 500003, FP32)])
@pytest.mark.parametrize("spread", [1e-1, 1e-3, 1e-4, 1e-5])
def test_kl_term_of_a_policy_next_to_its_reference(N, V, dtype, spread):
    """The term alone (no advantage).  With d = ref - logp known to within e, exp(d) - d - 1 is within
    |exp(d) - 1| e + e^2 of the exact one and its own rounding is relative to its own size; it is never negative."""
    i = policy_inputs(N + V, N, V, dtype, masked=0.0)
    z = i["logits"].double()
    logp = z.gather(1, i["targets"][:, None])[:, 0] - torch.logsumexp(z, 1)
    i["ref_logp"] = (logp + spread * randn(gen(5), N)).float()
    i["old_logp"] = logp.float()
    i["advantage"] = torch.zeros(N, device=DEV)
    row = policy(i, grad=False, kl_coef=1.0)[1]
    d = i["ref_logp"].double() - logp
    exact = torch.expm1(d) - d
    # e in units of 2^-24: the terms' arguments and ex2.approx (8), their additions along a lane (at most V / 256)
    # and across lanes and warps with their rescaling (28), the logarithm's own (4)
    e = EPS * (40 + V / 256)
    within(row, exact, torch.expm1(d).abs() * e + e * e + 16 * EPS * exact)
    assert bool((row >= 0).all())


# ----------------------------------------------------------------- in place

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 3, 7), (33, 8, 256), (9, 32, 1000), (77, 6, 130)])
@pytest.mark.parametrize("norm", [True, False])
def test_route_backward_in_place(T, k, E, norm):
    """dlogits may be the logits: the same bits."""
    g = gen(T + E)
    z = randn(g, T, E, std=3.0)
    top, idx = torch.topk(z, k, dim=1)
    idx = idx.int().contiguous()
    w = (torch.softmax(top, 1) if norm else torch.softmax(z, 1).gather(1, idx.long())).contiguous()
    dw, apart = randn(g, T, k), torch.empty(T, E, device=DEV)
    ftmoe.ftmoe_route_backward(z, idx, w, dw, T, E, k, norm, apart)
    ftmoe.ftmoe_route_backward(z, idx, w, dw, T, E, k, norm, z)
    assert torch.equal(z, apart)


# ----------------------------------------------------------------- the status word

def test_status_loses_no_mark_of_another_stream():
    """One thread reads and clears the word on a stream of its own while marks come from another stream: each
    mark shows in a read that had not returned when it was made."""
    table, out = torch.zeros(4, 8, device=DEV), torch.zeros(1, 8, device=DEV)
    bad = torch.full((1,), 9, device=DEV)
    reader, writer = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    stop, reads = threading.Event(), [0, 0]  # reads that returned, and those that saw a mark

    def read():
        while not stop.is_set():
            if ftmoe.ftmoe_ops_status(reader) == -10:
                reads[1] += 1
            reads[0] += 1

    thread = threading.Thread(target=read)
    thread.start()
    lost = 0
    try:
        for _ in range(2000):
            seen = reads[1]
            ftmoe.ftmoe_embed(table, 4, 8, bad, 1, 1.0, out, stream=writer)
            writer.synchronize()  # the mark is made
            done = reads[0]
            while reads[0] < done + 2 and thread.is_alive():  # a whole read has begun and returned since
                time.sleep(0)  # the other thread's turn
            lost += reads[1] == seen
    finally:
        stop.set()
        thread.join()
    assert lost == 0


# ----------------------------------------------------------------- AdamW: gradients that are not finite

@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_gradient_that_is_not_finite(value, bits):
    """NaN spoils its own value; an infinity does too, and in 8 bits the states of its block of 256.  Other
    blocks keep every bit."""
    n, at = 700, 300
    g = gen(3)

    def tensors(v):
        t = dict(p=randn(gen(4), n), g=randn(gen(5), n, std=0.1))
        if bits == 32:
            t.update(m=torch.zeros(n, device=DEV), v=torch.zeros(n, device=DEV))
        else:
            t.update(m=torch.zeros(n, dtype=torch.uint8, device=DEV), v=torch.zeros(n, dtype=torch.uint8, device=DEV),
                     m_scale=torch.zeros(3, device=DEV), v_scale=torch.zeros(3, device=DEV))
        if v is not None:
            t["g"][at] = v
        for step in (1, 2):
            ftmoe.ftmoe_adamw(ftmoe.adamw_list([t]), lr=1e-2, beta2=0.95, step=step)
            t["g"].copy_(randn(gen(5 + step), n, std=0.1))
        return t["p"]

    clean, dirty = tensors(None), tensors(value)
    same = torch.ones(n, dtype=torch.bool, device=DEV)
    same[at] = False
    assert not bool(torch.isfinite(dirty[at]))
    if bits == 8 and value != value or bits == 32:
        if bits == 8:  # the block's largest is taken of the other values, which may move a code
            same[256:512] = False
            rest = torch.arange(n, device=DEV)
            rest = rest[(rest >= 256) & (rest < 512) & (rest != at)]
            assert bool(torch.isfinite(dirty[rest]).all())
    else:
        same[256:512] = False
        assert bool(torch.isnan(dirty[256:512]).all())
    assert torch.equal(dirty[same], clean[same])


# ----------------------------------------------------------------- variants that other sizes do not reach

@pytest.mark.parametrize("T,k,H,dtype", [
    (130, 9, 2560, BF16), (400, 3, 2560, BF16), (700, 8, 2560, BF16), (700, 3, 1284, FP32), (1300, 2, 2560, FP16),
    (130, 3, 1001, BF16), (400, 2, 1001, FP32), (1300, 3, 1001, FP16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_combine_backward_of_one_to_eight_warps_a_token(T, k, H, dtype, in_place):
    base.test_combine_backward(T, k, 12, H, dtype, 0.3, in_place)


@pytest.mark.parametrize("T,k", [(2047, 1), (1024, 2), (256, 8), (683, 3), (2049, 1), (1025, 2), (257, 8), (32768, 1),
                                 (4097, 8)])
def test_dispatch_around_its_limits(T, k):
    """2048 pairs are the last that one launch counts, 32768 the last of the smaller sort."""
    base.test_dispatch(T, k, 40, 8, BF16, 0.1)


@pytest.mark.parametrize("N,V,dtype", [(5, 900001, BF16), (3, 1048576, FP16), (70, 450000, FP32)])
def test_policy_loss_of_rows_read_twice(N, V, dtype):
    i = policy_inputs(N + V, N, V, dtype, masked=0.3)
    kw = dict(temperature=0.9, kl_coef=0.05, clip_high=0.3)
    policy_check(i, policy(i, **kw), dtype, **kw)
    apart = policy(i, ld_d=V + 5, **kw)
    inp = policy(i, in_place=True, **kw)  # last: it overwrites the logits
    assert torch.equal(apart[3], inp[3]) and torch.equal(apart[0], inp[0])


# ----------------------------------------------------------------- policy loss: a wait that runs out

@pytest.mark.parametrize("N,V,dtype", [
    (16384, 65, FP32), (700, 130, BF16),           # a warp a row, several rows or one
    (1300, 4500, BF16), (300, 16001, FP16),        # two and four warps
    (300, 131072, BF16), (700, 50001, FP32), (3, 131072, BF16), (1, 20000, BF16)])
@pytest.mark.parametrize("grad", [True, False])
def test_policy_loss_wait_that_runs_out(N, V, dtype, grad):
    """A chunk is never asked for: its wait ends after 2 ms, the call reports it, rows come out as they should or
    as NaN, and the next call is as good as new."""
    i = policy_inputs(N + V, N, V, dtype, masked=0.3)
    i["weight"][0] = 1.0 / N
    want = policy(i, grad=grad, kl_coef=0.1)
    assert ftmoe.ftmoe_ops_status() == 0
    ftmoe.ftmoe_test_withhold_policy(True, 2_000_000)
    try:
        got = policy(i, grad=grad, kl_coef=0.1)
    finally:
        ftmoe.ftmoe_test_withhold_policy(False)
    assert ftmoe.ftmoe_ops_status() == -7 and ftmoe.ftmoe_ops_status() == 0
    assert bool(torch.isnan(got[0]).all())
    rows = [(g.view(N, -1), w.view(N, -1)) for g, w in zip(got[1:], want[1:]) if w is not None]
    same = torch.stack([(g == w).all(1) for g, w in rows]).all(0)
    lost = torch.stack([torch.isnan(g).all(1) for g, _ in rows]).all(0)
    assert bool((same ^ lost).all())
    assert bool(lost[0]) and (N < 300 or bool(same.any()))
    again = policy(i, grad=grad, kl_coef=0.1)
    assert ftmoe.ftmoe_ops_status() == 0
    assert all(torch.equal(a, w) for a, w in zip(again, want) if w is not None)


# ----------------------------------------------------------------- streams

def test_calls_without_a_stream_take_the_current_one():
    assert ftmoe._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert ftmoe._stream(None) == side.cuda_stream != 0
    assert ftmoe._stream(side) == side.cuda_stream
