"""Cases that measure a MoE layer on banks of 8-bit codes, from the router's logits to the experts' products.

Four operators: routing (softmax or sigmoid scores, a bias for balance,
groups, top-k) with its gradient; the quantiser of activations with a scale
for 128 values, which places tokens in expert order; the product of E4M3
codes with a scale for each block of 128, grouped by expert, with its SwiGLU
epilogue and the gradient of its input; SwiGLU between the products, with its
gradient.  Each case's ``run`` is one pass: the library's own calls when
``own`` is true, else the same mathematics in elementary torch operations.
``exact`` is the definition in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
BLOCK = 128  # values that share one scale; of weights a block of 128 x 128 does
TINY = 1e-30  # blocks whose largest value is below this are held as zeros
SKEW = 0.8  # expert of rank r is chosen in proportion to r^-SKEW


def listed():
    layer = dict(top_k=8, E=256, H=2560, I=640)  # the MoE layer's own sizes
    plain = dict(score="softmax", bias=False, n_groups=1, top_groups=1, group_best=1, norm=True)
    balanced = dict(score="sigmoid", bias=True, n_groups=8, top_groups=4, group_best=2, norm=True)
    return [
        # one decode step's tokens: latency
        dict(name="route_decode", op="route", T=16, E=256, top_k=8, dtype="fp32", grad=False, **plain),
        # the prefill batch, balanced by a bias, experts in eight groups of which a token takes four
        dict(name="route_groups", op="route", T=16384, E=256, top_k=8, dtype="fp32", grad=False, **balanced),
        # its gradient in a training batch
        dict(name="route_backward", op="route", T=16384, E=256, top_k=8, dtype="bf16", grad=True, **balanced),
        # a ragged batch on one rank of several: a quarter of the slots belong to other ranks, the last block is short
        dict(name="quantize_ragged", op="quantize", T=1023, top_k=6, E=60, H=2000, dtype="fp32", drop=True),
        # the prefill batch's tokens quantised into their experts' rows
        dict(name="quantize_prefill", op="quantize", T=16384, top_k=8, E=256, H=2560, dtype="bf16", drop=False),
        # one decode step through gate_up and SwiGLU: the touched experts' codes are read once
        dict(name="gate_up_decode", op="matmul", T=16, product="gate_up", swiglu=True, dtype="bf16", **layer),
        # one token through down: fewer tiles than SMs
        dict(name="down_one_token", op="matmul", T=1, product="down", swiglu=False, dtype="fp32", **layer),
        # the prefill batch through gate_up and SwiGLU
        dict(name="gate_up_prefill", op="matmul", T=16384, product="gate_up", swiglu=True, dtype="bf16", **layer),
        # few experts of odd widths, output in 32 bits
        dict(name="matmul_ragged", op="matmul", T=1023, top_k=6, E=60, H=2000, I=333, product="gate_up", swiglu=False,
             dtype="fp32"),
        # a training batch's gradient through gate_up to its input
        dict(name="gate_up_input_grad", op="matmul", T=16384, product="gate_up_grad", swiglu=False, dtype="bf16",
             **layer),
        # a training batch between the products, quantised for the next one
        dict(name="swiglu_batch", op="swiglu", rows=131072, I=640, dtype="bf16", codes=True, grad=False),
        # its gradient, of an odd width, kept in 16 bits
        dict(name="swiglu_backward_odd", op="swiglu", rows=8191, I=1001, dtype="fp16", codes=False, grad=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "matmul", "matmul", "swiglu"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "route":
        gs, n = _log_int(rng, 2, 64), rng.choice([1, 1, 2, 4, 7, 8, 16])
        E = _log_int(rng, 2, 1024) if n == 1 else gs * n
        top_groups = rng.randint(1, n)
        k = rng.randint(1, min(16, E // n * top_groups))
        return dict(op=op, T=_log_int(rng, 1, min(16384, 16384 * 256 // E)), E=E, top_k=k, dtype=dtype,
                    grad=rng.random() < 0.4, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    n_groups=n, top_groups=top_groups, group_best=rng.choice([1, 2]) if n > 1 else 1,
                    norm=rng.random() < 0.7)
    if op == "swiglu":
        codes = rng.random() < 0.6
        I = _log_int(rng, 64, 8192)
        if codes:
            I = max(128, I // 128 * 128)
        return dict(op=op, rows=_log_int(rng, 1, max(1, min(131072, 131072 * 640 * 2 // (I * SIZE[dtype])))), I=I,
                    dtype=dtype, codes=codes, grad=rng.random() < 0.5)
    H = 16 * _log_int(rng, 4, 512)
    if op == "quantize":
        E = _log_int(rng, 2, 1024)
        k = rng.randint(1, min(E, 16))
        T = _log_int(rng, 1, max(1, min(16384, 16384 * 8 * 2560 // (H * k))))
        return dict(op=op, T=T, top_k=k, E=E, H=H, dtype=dtype, drop=rng.random() < 0.5)
    product = rng.choice(["gate_up", "gate_up", "down", "gate_up_grad"])
    swiglu = product == "gate_up" and rng.random() < 0.6
    I = 128 * _log_int(rng, 1, 32) if swiglu else 16 * _log_int(rng, 4, 256)
    E = _log_int(rng, 1, max(1, min(512, 256 * 640 * 2560 // (I * H))))
    k = rng.randint(1, min(E, 16))
    T = _log_int(rng, 1, max(1, min(16384, 16384 * 8 * 640 * 2560 // (k * I * H), 16384 * 8 * 2560 // (k * max(H, 2 * I)))))
    return dict(op=op, T=T, top_k=k, E=E, H=H, I=I, product=product, swiglu=swiglu,
                dtype="bf16" if swiglu else rng.choice(["bf16", "bf16", "fp16", "fp32"]))


# ----------------------------------------------------------------- inputs

def _experts(case, g, dev):
    """Distinct experts per token, those of low rank more often: [T, top_k] int32."""
    T, k, E = case["T"], case["top_k"], case["E"]
    prior = -SKEW * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    prior = prior[torch.randperm(E, generator=g, device=dev)]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev).clamp(1e-7, 1 - 1e-7)))
    return torch.topk(noise + prior, k, dim=1).indices.int()


def _touched(case):
    """Experts that a batch is expected to reach."""
    p = [r ** -SKEW for r in range(1, case["E"] + 1)]
    return sum(1 - (1 - min(1.0, case["top_k"] * x / sum(p))) ** case["T"] for x in p)


def _sizes(case):
    """(N, K) of an expert's matrix [N, K] of a product case, and the lengths of its input's and output's rows."""
    H, I = case["H"], case["I"]
    N, K = (H, I) if case["product"] == "down" else (2 * I, H)
    if case["product"] == "gate_up_grad":
        return N, K, N, K
    return N, K, K, N // 2 if case["swiglu"] else N


def _blocks(n):
    return -(-n // BLOCK)


def _quantized(x):
    """Codes of x [rows, n] with a scale for 128 values, and the scales [ceil(n / 128), rows]."""
    rows, n = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _blocks(n) * BLOCK - n)).view(rows, -1, BLOCK)
    top = x.abs().amax(2, keepdim=True)
    scale = torch.where(top < TINY, 0.0, top / 448)
    codes = torch.where(top < TINY, 0.0, x * (448 / top)).to(E4M3).view(rows, -1)[:, :n]
    return codes.contiguous(), scale[:, :, 0].t().contiguous()


def _spread(scale, n, dim):
    """Each scale along `dim` for its 128 values, n in all."""
    return scale.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    if op == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        s.update(logits=randn(T, E).to(dt), b=randn(E, std=0.1) if case["bias"] else None, scale=2.5,
                 idx=torch.empty(T, k, dtype=torch.int32, device=dev), w=torch.empty(T, k, device=dev))
        if case["grad"]:
            s["idx"], s["w"] = _route_plain(s)
            s.update(dw=randn(T, k, std=0.05), dlogits=torch.empty(T, E, dtype=dt, device=dev))
        return s
    if op == "quantize":
        T, k, H = case["T"], case["top_k"], case["H"]
        idx = _experts(case, g, dev)
        if case["drop"]:
            idx = torch.where(torch.rand(T, k, generator=g, device=dev) < 0.25, -1, idx)
        key = torch.where(idx < 0, case["E"], idx).view(-1)
        order = torch.argsort(key, stable=True)
        inv = torch.empty_like(order)
        inv[order] = torch.arange(T * k, device=dev)
        # tokens and single channels differ in size
        x = randn(T, H) * torch.exp(0.5 * randn(T, 1)) * torch.exp(0.5 * randn(1, H))
        s.update(x=x.to(dt), inv=torch.where(key < case["E"], inv, -1).int(),
                 codes=torch.zeros(T * k, H, dtype=torch.uint8, device=dev).view(E4M3),
                 scales=torch.zeros(_blocks(H), T * k, device=dev))
        return s
    if op == "swiglu":
        n, I = case["rows"], case["I"]
        s.update(gu=randn(n, 2 * I).to(dt), dh=randn(n, I, std=0.05).to(dt) if case["grad"] else None)
        width = 2 * I if case["grad"] else I
        s.update(out=torch.empty(n, width, dtype=E4M3 if case["codes"] else dt, device=dev),
                 scales=torch.empty(_blocks(width), n, device=dev) if case["codes"] else None)
        return s
    E, P = case["E"], case["T"] * case["top_k"]
    N, K, width, out_width = _sizes(case)
    counts = torch.bincount(_experts(case, g, dev).view(-1), minlength=E)
    offsets = torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).int()
    codes = torch.empty(E, N, K, dtype=E4M3, device=dev)
    scales = torch.empty(E, _blocks(N), _blocks(K), device=dev)
    for e in range(E):  # expert by expert: a bank in 32 bits is four times its codes
        w = torch.nn.functional.pad(randn(N, K, std=0.02), (0, _blocks(K) * BLOCK - K, 0, _blocks(N) * BLOCK - N))
        w = w.view(_blocks(N), BLOCK, _blocks(K), BLOCK)
        top = w.abs().amax((1, 3), keepdim=True)
        codes[e] = (w * (448 / top)).to(E4M3).view(_blocks(N) * BLOCK, -1)[:N, :K]
        scales[e] = top[:, 0, :, 0] / 448
    a = randn(P, width) * torch.exp(0.5 * randn(P, 1))
    s["a"], s["a_scale"] = _quantized(a)
    s.update(weights=codes, w_scale=scales, offsets=offsets, bounds=offsets.tolist(),
             out=torch.empty(P, out_width, dtype=E4M3 if case["swiglu"] else dt, device=dev),
             out_scale=torch.empty(_blocks(out_width), P, device=dev) if case["swiglu"] else None)
    return s


# ----------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from nvfp4_mixture_experts_counting_gb300 import ftmoe
    op = s["op"]
    if op == "route":
        a = ftmoe.route_args(s["logits"], s["idx"], s["w"], score=s["score"], norm_topk_prob=s["norm"],
                             scale=s["scale"], bias=s["b"], n_groups=s["n_groups"], top_groups=s["top_groups"],
                             group_best=s["group_best"])
        if s["grad"]:
            ftmoe.ftmoe_route_topk_backward(a, s["dw"], s["dlogits"])
            return [s["dlogits"]]
        ftmoe.ftmoe_route_topk(a)
        return [s["idx"], s["w"]]
    if op == "quantize":
        ftmoe.ftmoe_fp8_quantize(s["x"], s["T"], s["H"], s["inv"], s["top_k"], s["codes"], s["scales"])
        return [s["codes"], s["scales"]]
    if op == "swiglu":
        if s["grad"]:
            ftmoe.ftmoe_swiglu_backward(s["dh"], s["gu"], s["rows"], s["I"], s["out"], s["scales"])
        else:
            ftmoe.ftmoe_swiglu(s["gu"], s["rows"], s["I"], s["out"], s["scales"])
        return [s["out"], s["scales"]] if s["codes"] else [s["out"]]
    N, K, _, _ = _sizes(s)
    ftmoe.ftmoe_fp8_matmul(s["a"], s["a_scale"], s["weights"], s["w_scale"], s["offsets"], s["T"] * s["top_k"], s["E"],
                           N, K, s["out"], s["out_scale"], transpose=s["product"] == "gate_up_grad",
                           swiglu=s["swiglu"])
    return [s["out"], s["out_scale"]] if s["swiglu"] else [s["out"]]


def _route_plain(s):
    """Chosen experts and their weights; scores in 64 bits, where neighbours in rank stay apart."""
    z = s["logits"].double()
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) if s["score"] == "softmax" else 1 / (1 + torch.exp(-z))
    c = p if s["b"] is None else p + s["b"].double()
    if s["n_groups"] > 1:
        members = c.view(c.shape[0], s["n_groups"], -1)
        best = torch.sort(members, dim=2, descending=True).values[:, :, :s["group_best"]].sum(2)
        groups = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        on = torch.zeros_like(best).scatter_(1, groups, 1.0)
        c = torch.where(on[:, :, None] > 0, members, -math.inf).view_as(c)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    w = p.gather(1, idx)
    if s["norm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (w * s["scale"]).float()


def _run_plain(s):
    op = s["op"]
    if op == "route":
        if not s["grad"]:
            return list(_route_plain(s))
        z, at, w = s["logits"].float(), s["idx"].long(), s["w"]
        D = (w * s["dw"]).sum(1, keepdim=True)
        up = s["dw"] - D / s["scale"] if s["norm"] else s["dw"]
        if s["score"] == "sigmoid":
            d = torch.zeros_like(z).scatter_(1, at, w * up / (1 + torch.exp(z.gather(1, at))))
        elif s["norm"]:
            d = torch.zeros_like(z).scatter_(1, at, w * up)
        else:
            e = torch.exp(z - z.amax(1, keepdim=True))
            d = e / e.sum(1, keepdim=True) * (torch.zeros_like(z).scatter_(1, at, s["dw"] * s["scale"]) - D)
        return [d.to(s["dlogits"].dtype)]
    if op == "quantize":
        codes, scales = _quantized(s["x"])
        P, k, H = s["inv"].numel(), s["top_k"], s["H"]
        to = torch.where(s["inv"] >= 0, s["inv"], P).long()  # the last row takes what is dropped
        out = torch.zeros(P + 1, H, dtype=torch.uint8, device=to.device)
        out[to] = codes.view(torch.uint8)[torch.arange(P, device=to.device) // k]
        placed = torch.zeros(scales.shape[0], P + 1, device=to.device)
        placed[:, to] = scales.repeat_interleave(k, 1)
        return [out[:P].view(E4M3), placed[:, :P].contiguous()]
    if op == "swiglu":
        g, u = s["gu"].float().chunk(2, 1)
        sig = 1 / (1 + torch.exp(-g))
        if s["grad"]:
            dh = s["dh"].float()
            out = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
        else:
            out = g * sig * u
        return list(_quantized(out)) if s["codes"] else [out.to(s["out"].dtype)]
    N, K, width, _ = _sizes(s)
    a = s["a"].float() * _spread(s["a_scale"].t(), width, 1)
    y = torch.empty(a.shape[0], K if s["product"] == "gate_up_grad" else N, device=a.device)
    for e in range(s["E"]):  # a product for each expert, as a program without a grouped one has them
        rows = slice(s["bounds"][e], s["bounds"][e + 1])
        if rows.start < rows.stop:
            w = s["weights"][e].float() * _spread(_spread(s["w_scale"][e], N, 0), K, 1)
            torch.matmul(a[rows], w if s["product"] == "gate_up_grad" else w.t(), out=y[rows])
    if not s["swiglu"]:
        return [y.to(s["out"].dtype)]
    g, u = y.chunk(2, 1)
    return list(_quantized(g / (1 + torch.exp(-g)) * u))


def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        if not case["grad"]:
            return {"bytes": T * E * b + T * k * 8 + E * 4 * case["bias"], "flops": 4 * T * E}
        read = T * E * b if case["score"] == "softmax" and not case["norm"] else 0
        return {"bytes": read + T * E * b + T * k * (12 + (b if case["score"] == "sigmoid" else 0)), "flops": T * E}
    if op == "quantize":
        T, P, H = case["T"], case["T"] * case["top_k"], case["H"]
        kept = 0.75 * P if case["drop"] else P
        return {"bytes": int(T * H * b + kept * (H + 4 * _blocks(H)) + 4 * P), "flops": 3 * T * H}
    if op == "swiglu":
        n, I = case["rows"], case["I"]
        width = 2 * I if case["grad"] else I
        out = n * (width + 4 * _blocks(width)) if case["codes"] else n * width * b
        return {"bytes": n * I * (3 if case["grad"] else 2) * b + out, "flops": (12 if case["grad"] else 6) * n * I}
    P, (N, K, width, out_width) = case["T"] * case["top_k"], _sizes(case)
    out = P * (out_width + 4 * _blocks(out_width)) if case["swiglu"] else P * out_width * b
    weights = _touched(case) * (N * K + 4 * _blocks(N) * _blocks(K))
    return {"bytes": int(weights + P * (width + 4 * _blocks(width)) + out), "flops": 2 * P * N * K}


# ----------------------------------------------------------------- the definition in 64 bits

def _codes_of(x):
    """E4M3 codes and scales of x [rows, n] in 64 bits, a scale for 128 values."""
    rows, n = x.shape
    blocks = torch.split(x, BLOCK, 1)
    scale = torch.stack([p.abs().amax(1) / 448 for p in blocks])
    codes = torch.cat([p / torch.where(f > 0, f, 1.0)[:, None] for p, f in zip(blocks, scale)], 1)
    return codes.to(E4M3).double(), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        z, k = s["logits"].double(), case["top_k"]
        prob = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
        if case["grad"]:
            at = s["idx"].long()
            p = prob.detach().gather(1, at)
            w = s["scale"] * (p / p.sum(1, keepdim=True) if case["norm"] else p)
            dw = s["dw"].double()
            # d w_j / d s_i, then d s_i / d z_e
            ds = dw * s["scale"]
            if case["norm"]:
                ds = (ds - (ds * p).sum(1, keepdim=True) / p.sum(1, keepdim=True)) / p.sum(1, keepdim=True)
            full = torch.zeros_like(z).scatter_add_(1, at, ds)
            if case["score"] == "sigmoid":
                return [full * prob * (1 - prob)]
            return [prob * (full - (full * prob).sum(1, keepdim=True))]
        rank = prob + (s["b"].double() if case["bias"] else 0.0)
        if case["n_groups"] > 1:
            by = rank.view(case["T"], case["n_groups"], -1)
            value = torch.topk(by, case["group_best"], 2).values.sum(2)
            keep = torch.argsort(value, dim=1, descending=True, stable=True).argsort(dim=1) < case["top_groups"]
            rank = rank.masked_fill(~keep.repeat_interleave(by.shape[2], 1), -math.inf)
        idx = torch.argsort(rank, dim=1, descending=True, stable=True)[:, :k]
        w = torch.take_along_dim(prob, idx, 1)
        if case["norm"]:
            w = w / w.sum(1, keepdim=True)
        return [idx.int(), s["scale"] * w]
    if op == "quantize":
        codes, scale = _codes_of(s["x"].double())
        P = case["T"] * case["top_k"]
        out = torch.zeros(P, case["H"], dtype=torch.float64, device="cuda")
        placed = torch.zeros(_blocks(case["H"]), P, dtype=torch.float64, device="cuda")
        inv = s["inv"].view(case["T"], case["top_k"]).long()
        for j in range(case["top_k"]):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            out[inv[t, j]] = codes[t]
            placed[:, inv[t, j]] = scale[:, t]
        return [out, placed]
    if op == "swiglu":
        g, u = s["gu"][:, :case["I"]].double(), s["gu"][:, case["I"]:].double()
        if case["grad"]:
            d, sig = s["dh"].double(), torch.sigmoid(g)
            out = torch.cat([d * u * (sig + g * sig * (1 - sig)), d * torch.nn.functional.silu(g)], 1)
        else:
            out = torch.nn.functional.silu(g) * u
        return list(_codes_of(out)) if case["codes"] else [out]
    N, K, width, out_width = _sizes(case)
    back = case["product"] == "gate_up_grad"
    P = s["a"].shape[0]
    y = torch.zeros(P, K if back else N, dtype=torch.float64, device="cuda")
    at = torch.arange(max(N, K), device="cuda") // BLOCK
    for e, (i, j) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        if i < j:
            w = s["weights"][e].double() * s["w_scale"][e].double()[at[:N]][:, at[:K]]
            x = s["a"][i:j].double() * s["a_scale"][:, i:j].double()[at[:width]].t()
            y[i:j] = torch.einsum("rn,nk->rk" if back else "rk,nk->rn", x, w)
    if not case["swiglu"]:
        return [y]
    h = torch.nn.functional.silu(y[:, :case["I"]])
    h *= y[:, case["I"]:]
    return list(_codes_of(h))
