"""Cases that measure the operators of a training step around the MoE layer.

Four operators: tokens sorted by expert and back (dispatch, combine and their
gradients), the embedding lookup and its gradient, the clipped policy loss
with its KL term (forward and backward in one call), and the AdamW step over
a list of tensors.  Each case's ``run`` is one pass: the library's own calls
when ``own`` is true, else the same mathematics in elementary torch
operations in 32 bits.  ``exact`` is the definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
BLOCK = 256  # values that share one scale in the 8-bit optimiser state
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05
ADAM = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, step=7)
WEIGHT_DECAY = 0.1
GRAD_SCALE = 0.75  # what clipping the gradients to their norm leaves of them


def listed():
    layer = dict(top_k=8, E=256, H=2560)  # the MoE layer's own sizes
    return [
        # one decode step's tokens: the time is launches and latency
        dict(name="dispatch_decode", op="dispatch", T=16, dtype="bf16", drop=False, **layer),
        # the prefill batch: the copy of every token's row to its experts' rows
        dict(name="dispatch_prefill", op="dispatch", T=16384, dtype="bf16", drop=False, **layer),
        # a ragged batch on one rank of several: a quarter of the slots belong to other ranks
        dict(name="combine_ragged", op="combine", T=1023, dtype="fp32", drop=True, weighted=True,
             top_k=6, E=60, H=2000),
        # the gradient of a training batch down to the router's logits
        dict(name="combine_backward", op="combine_backward", T=16384, dtype="bf16", drop=False, norm=True, **layer),
        # the input of a training batch of 16384 tokens
        dict(name="embed_batch", op="embed", N=16384, V=131072, H=2560, dtype="bf16", wide_ids=True),
        # its gradient: few tokens make up much of the text, most rows get none
        dict(name="embed_backward", op="embed_backward", N=16384, V=131072, H=2560, dtype="bf16", table="bf16",
             wide_ids=True),
        # a small vocabulary with an odd width, gradients in 32 bits, every row hit many times
        dict(name="embed_backward_odd", op="embed_backward", N=8191, V=1000, H=1001, dtype="bf16", table="fp32",
             wide_ids=False),
        # a training batch's logits
        dict(name="policy_batch", op="policy_loss", N=4096, V=131072, dtype="bf16", masked=0.2, grad=True),
        # a few tokens: rows are fewer than the SMs
        dict(name="policy_few_rows", op="policy_loss", N=5, V=131072, dtype="bf16", masked=0.0, grad=True),
        # odd rows in 32 bits, whose starts share no alignment
        dict(name="policy_odd", op="policy_loss", N=1023, V=50001, dtype="fp32", masked=0.2, grad=True),
        # all tensors of 48 bf16 layers with master weights, states in 32 bits
        dict(name="adamw_stack", op="adamw", layers=48, H=2560, I=640, E=256, dtype="bf16", master=True, bits=32),
        # the same layers with states in 8 bits and no master weights
        dict(name="adamw_stack_8bit", op="adamw", layers=48, H=2560, I=640, E=256, dtype="bf16", master=False, bits=8),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n - (n == 3072)))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_backward", "embed", "embed_backward", "policy_loss", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    H = _log_int(rng, 64, 8192)
    if rng.random() < 0.8:
        H = max(16, H // 16 * 16 + (16 if H // 16 == 192 else 0))
    if op in ("dispatch", "combine", "combine_backward"):
        E = _log_int(rng, 2, 1024)
        k = rng.randint(1, min(E, 16))
        T = _log_int(rng, 1, max(1, min(16384, 16384 * 8 * 2560 * 2 // (H * k * SIZE[dtype]))))
        c = dict(op=op, T=T, top_k=k, E=E, H=H, dtype=dtype, drop=rng.random() < 0.5)
        if op == "combine":
            c["weighted"] = rng.random() < 0.5
        if op == "combine_backward":
            c["norm"] = rng.random() < 0.5
        return c
    if op == "embed":
        V = _log_int(rng, 2, min(262144, 131072 * 2560 * 2 // (H * SIZE[dtype])))
        N = _log_int(rng, 1, max(1, min(65536, 65536 * 2560 * 2 // (H * SIZE[dtype]))))
        return dict(op=op, N=N, V=V, H=H, dtype=dtype, wide_ids=rng.random() < 0.5)
    if op == "embed_backward":
        table = rng.choice([dtype, "fp32"])
        V = _log_int(rng, 2, max(2, min(262144, 131072 * 2560 * 2 // (H * SIZE[table]))))
        N = _log_int(rng, 1, max(1, min(65536, 65536 * 2560 * 2 // (H * SIZE[dtype]))))
        return dict(op=op, N=N, V=V, H=H, dtype=dtype, table=table, wide_ids=rng.random() < 0.5)
    if op == "policy_loss":
        V = _log_int(rng, 100, 200000)
        N = _log_int(rng, 1, max(1, min(16384, 4096 * 131072 * 2 // (V * SIZE[dtype]))))
        return dict(op=op, N=N, V=V, dtype=dtype, masked=rng.choice([0.0, 0.2, 0.6]), grad=rng.random() < 0.75)
    I = max(1, H // 4 + rng.randint(-8, 8))
    E = _log_int(rng, 2, 512)
    per_layer = E * H + 3 * I * H + H + E + 1
    layers = _log_int(rng, 1, max(1, min(48, 250_000_000 // per_layer)))
    return dict(op=op, layers=layers, H=H, I=I, E=E, dtype=dtype, master=dtype != "fp32" and rng.random() < 0.5,
                bits=rng.choice([8, 32]))


# ----------------------------------------------------------------- inputs

def _experts(case, g, dev):
    """Distinct experts per token under a skewed prior; dropped slots are -1."""
    T, k, E = case["T"], case["top_k"], case["E"]
    prior = -0.8 * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    prior = prior[torch.randperm(E, generator=g, device=dev)]
    logits = torch.randn(T, E, generator=g, device=dev) + prior
    top, idx = torch.topk(logits, k, dim=1)
    kept = idx.int()
    if case["drop"]:
        kept = torch.where(torch.rand(T, k, generator=g, device=dev) < 0.25, -1, kept)
    return logits, idx.int(), kept.contiguous(), torch.softmax(top, 1)


def _sorted_places(kept, E):
    """inv of the stable sort by expert, -1 where dropped."""
    key = torch.where((kept < 0) | (kept >= E), E, kept).reshape(-1)
    order = torch.argsort(key, stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(order.numel(), device=order.device)
    return torch.where(key < E, inv, -1).int()


def _ids(case, g, dev):
    """Token ids whose frequency falls as one over their rank, ranks spread over the vocabulary."""
    V = case["V"]
    rank = torch.exp(torch.rand(case["N"], generator=g, device=dev, dtype=torch.float64) * math.log(V)).long() - 1
    ids = (rank.clamp(0, V - 1) * 1000003 + 17) % V
    return ids if case["wide_ids"] else ids.int()


def _adam_shapes(case):
    H, I, E = case["H"], case["I"], case["E"]
    return [(E * H, True), (2 * I * H, True), (H * I, True), (H, False), (E, False), (1, False)] * case["layers"]


def _adam_places(case):
    """(start, size, decayed) of each tensor in the flat buffers: each starts on a multiple of BLOCK."""
    at, places = 0, []
    for n, decayed in _adam_shapes(case):
        places.append((at, n, decayed))
        at += -(-n // BLOCK) * BLOCK
    return places, at


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    if op in ("dispatch", "combine", "combine_backward"):
        T, k, E, H = case["T"], case["top_k"], case["E"], case["H"]
        P = T * k
        logits, idx, kept, w = _experts(case, g, dev)
        if op == "dispatch":
            s.update(x=randn(T, H), idx=kept, offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                     perm=torch.empty(P, dtype=torch.int32, device=dev),
                     inv=torch.empty(P, dtype=torch.int32, device=dev),
                     xs=torch.zeros(P, H, dtype=dt, device=dev))
            return s
        s.update(ys=randn(P, H), inv=_sorted_places(kept, E), w=w)
        if op == "combine":
            s["out"] = torch.empty(T, H, dtype=dt, device=dev)
            return s
        if not case["norm"]:
            s["w"] = torch.gather(torch.softmax(logits, 1), 1, idx.long())
        s.update(dout=randn(T, H, std=0.05), logits=logits, idx=idx, dys=torch.zeros(P, H, dtype=dt, device=dev),
                 dw=torch.empty(T, k, device=dev), dlogits=torch.empty(T, E, device=dev))
        return s
    if op in ("embed", "embed_backward"):
        N, V, H = case["N"], case["V"], case["H"]
        s.update(ids=_ids(case, g, dev), scale=math.sqrt(H))
        if op == "embed":
            s.update(weights=randn(V, H, std=0.02), out=torch.empty(N, H, dtype=dt, device=dev))
        else:
            s.update(dout=randn(N, H, std=0.05), dtable=torch.empty(V, H, dtype=DTYPES[case["table"]], device=dev))
        return s
    if op == "policy_loss":
        N, V = case["N"], case["V"]
        logits = torch.empty(N, V, dtype=dt, device=dev)
        for i in range(0, N, 1024):
            logits[i:i + 1024] = randn(min(1024, N - i), V, std=2.0)
        targets = torch.randint(0, V, (N,), generator=g, device=dev)
        targets[::2] = logits[::2].argmax(1)  # what a policy samples is mostly likely
        logp = torch.cat([torch.log_softmax(logits[i:i + 256].float(), 1).gather(1, targets[i:i + 256, None])[:, 0]
                          for i in range(0, N, 256)])
        keep = (torch.rand(N, generator=g, device=dev) >= case["masked"]).float()
        s.update(logits=logits, targets=targets, old=logp + 0.2 * torch.randn(N, generator=g, device=dev),
                 ref=logp + 0.3 * torch.randn(N, generator=g, device=dev),
                 adv=torch.randn(N, generator=g, device=dev), weight=keep / keep.sum().clamp(min=1),
                 loss=torch.empty(1, device=dev), row_loss=torch.empty(N, device=dev),
                 logp=torch.empty(N, device=dev), dlogits=torch.empty_like(logits) if case["grad"] else None)
        return s
    places, total = _adam_places(case)
    real = torch.zeros(total // BLOCK, BLOCK, dtype=torch.bool, device=dev)
    decay = torch.zeros(total // BLOCK, 1, device=dev)
    for at, n, decayed in places:
        real.view(-1)[at:at + n] = True
        decay[at // BLOCK:(at + n + BLOCK - 1) // BLOCK] = WEIGHT_DECAY if decayed else 0.0
    # tensors' gradients differ in size, and the values of one block do too
    size = torch.exp(torch.randn(total // BLOCK, 1, generator=g, device=dev))

    def values(std):
        return torch.randn(total // BLOCK, BLOCK, generator=g, device=dev).mul_(std).mul_(real)

    master = values(0.02)
    m = values(1e-3).mul_(size)
    u = values(3e-3).mul_(size).abs_()
    s.update(grad=values(1e-2).mul_(size).to(dt).view(-1), p=master.to(dt).view(-1), decay=decay,
             grad_scale=torch.full((1,), GRAD_SCALE, device=dev), places=places,
             master=master.view(-1) if case["master"] else None)
    if case["bits"] == 32:
        s.update(m=m.view(-1), v=u.square_().view(-1))
        return s
    for name, x in (("m", m), ("v", u)):
        scale = (x.abs().amax(1) / 448).clamp(min=1e-20)
        s[name] = (x / scale[:, None]).to(E4M3).view(-1)
        s[name + "_scale"] = scale
    return s


# ----------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from nvfp4_mixture_experts_counting_gb300 import ftmoe
    op = s["op"]
    if op == "dispatch":
        ftmoe.ftmoe_dispatch(s["x"], s["T"], s["H"], s["idx"], s["top_k"], s["E"], s["offsets"], s["perm"], s["inv"],
                             s["xs"])
        return [s["offsets"], s["perm"], s["inv"], s["xs"]]
    if op == "combine":
        ftmoe.ftmoe_combine(s["ys"], s["T"], s["H"], s["top_k"], s["inv"], s["w"] if s["weighted"] else None, s["out"])
        return [s["out"]]
    if op == "combine_backward":
        ftmoe.ftmoe_combine_backward(s["dout"], s["ys"], s["T"], s["H"], s["top_k"], s["inv"], s["w"], s["dys"],
                                     s["dw"])
        ftmoe.ftmoe_route_backward(None if s["norm"] else s["logits"], s["idx"], s["w"], s["dw"], s["T"], s["E"],
                                   s["top_k"], s["norm"], s["dlogits"])
        return [s["dys"], s["dw"], s["dlogits"]]
    if op == "embed":
        ftmoe.ftmoe_embed(s["weights"], s["V"], s["H"], s["ids"], s["N"], s["scale"], s["out"])
        return [s["out"]]
    if op == "embed_backward":
        if "workspace" not in s:
            s["workspace"] = torch.empty(ftmoe.ftmoe_embed_workspace(s["N"], s["H"]), dtype=torch.uint8, device="cuda")
        ftmoe.ftmoe_embed_backward(s["dout"], s["ids"], s["N"], s["V"], s["H"], s["scale"], -1, s["dtable"], False,
                                   s["workspace"])
        return [s["dtable"]]
    if op == "policy_loss":
        a = ftmoe.policy_args(s["logits"], s["targets"], s["old"], s["ref"], s["adv"], s["weight"], s["loss"],
                              s["row_loss"], s["logp"], s["dlogits"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                              kl_coef=KL_COEF)
        ftmoe.ftmoe_policy_loss(a)
        return [s["loss"], s["row_loss"], s["logp"], s["dlogits"]]
    if "list" not in s:  # a training program lists its tensors once
        eight = s["bits"] == 8
        s["list"] = ftmoe.adamw_list([
            dict(p=s["p"][a:a + n], g=s["grad"][a:a + n], master=s["master"][a:a + n] if s["master"] is not None else None,
                 m=s["m"][a:a + n], v=s["v"][a:a + n],
                 m_scale=s["m_scale"][a // BLOCK:(a + n + BLOCK - 1) // BLOCK] if eight else None,
                 v_scale=s["v_scale"][a // BLOCK:(a + n + BLOCK - 1) // BLOCK] if eight else None,
                 weight_decay=WEIGHT_DECAY if decayed else 0.0) for a, n, decayed in s["places"]])
    ftmoe.ftmoe_adamw(s["list"], grad_scale=s["grad_scale"], **ADAM)
    return _adam_outputs(s)


def _adam_outputs(s):
    return {n: s[n] for n in ("p", "master", "m", "v", "m_scale", "v_scale") if s.get(n) is not None}


def _run_plain(s):
    op = s["op"]
    if op == "dispatch":
        E, k, P = s["E"], s["top_k"], s["T"] * s["top_k"]
        flat = s["idx"].reshape(-1)
        key = torch.where((flat < 0) | (flat >= E), E, flat)
        ordered, order = torch.sort(key, stable=True)
        place = torch.arange(P, device=key.device, dtype=torch.int32)
        offsets = torch.searchsorted(ordered, torch.arange(E + 1, device=key.device, dtype=torch.int32)).int()
        perm = torch.where(ordered < E, order, -1).int()
        inv = torch.empty_like(perm)
        inv[order] = torch.where(ordered < E, place, -1)
        xs = torch.where((ordered < E)[:, None], s["x"][order // k], 0)
        return [offsets, perm, inv, xs]
    if op == "combine":
        inv = s["inv"].view(s["T"], s["top_k"])
        rows = s["ys"][inv.clamp(min=0)].float()
        w = (inv >= 0).float() * (s["w"] if s["weighted"] else 1.0)
        return [(rows * w[:, :, None]).sum(1).to(s["ys"].dtype)]
    if op == "combine_backward":
        inv, w = s["inv"].view(s["T"], s["top_k"]), s["w"]
        kept = inv >= 0
        d = s["dout"].float()
        dw = (s["ys"][inv.clamp(min=0)].float() * d[:, None, :]).sum(2) * kept
        P = inv.numel()
        dys = torch.zeros(P + 1, s["H"], dtype=s["ys"].dtype, device=d.device)  # the last row takes what is dropped
        dys[torch.where(kept, inv, P).view(-1)] = (w[:, :, None] * d[:, None, :]).to(dys.dtype).view(P, -1)
        S = (w * dw).sum(1, keepdim=True)
        if s["norm"]:
            dl = torch.zeros_like(s["logits"])
            dl.scatter_add_(1, s["idx"].long(), w * (dw - S))
        else:
            e = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
            chosen = torch.zeros_like(s["logits"]).scatter_add_(1, s["idx"].long(), dw)
            dl = e / e.sum(1, keepdim=True) * (chosen - S)
        return [dys[:P], dw, dl]
    if op == "embed":
        return [(s["weights"][s["ids"].long()].float() * s["scale"]).to(s["weights"].dtype)]
    if op == "embed_backward":
        grad = torch.zeros(s["V"], s["H"], device=s["dout"].device)
        grad.index_add_(0, s["ids"].long(), s["dout"].float())
        return [(grad * s["scale"]).to(s["dtable"].dtype)]
    if op == "policy_loss":
        z = s["logits"].float()
        y = s["targets"][:, None]
        top = z.amax(1, keepdim=True)
        lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
        counted = s["weight"] != 0
        logp = torch.where(counted, (z.gather(1, y) - lse)[:, 0], 0.0)
        r, d = torch.exp(logp - s["old"]), s["ref"] - logp
        plain, clipped = r * s["adv"], r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * s["adv"]
        row = torch.where(counted, -torch.minimum(plain, clipped) + KL_COEF * (torch.exp(d) - d - 1), 0.0)
        loss = (s["weight"] * row).sum().view(1)
        if not s["grad"]:
            return [loss, row, logp, None]
        c = s["weight"] * (KL_COEF * (1 - torch.exp(d)) - torch.where(plain <= clipped, plain, 0.0))
        dz = torch.exp(z - lse) * -c[:, None]
        dz.scatter_add_(1, y, c[:, None])
        return [loss, row, logp, dz.to(s["logits"].dtype)]
    # AdamW, on all tensors' blocks at once
    b1, b2, t = ADAM["beta1"], ADAM["beta2"], ADAM["step"]
    g = s["grad"].view(-1, BLOCK).float() * s["grad_scale"]
    eight = s["bits"] == 8
    m, v = s["m"].view(-1, BLOCK).float(), s["v"].view(-1, BLOCK).float()
    if eight:
        m = m * s["m_scale"][:, None]
        v = v * s["v_scale"][:, None]
        v = v * v
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = torch.sqrt(v)
    update = m / (root * (1 / math.sqrt(1 - b2 ** t)) + ADAM["eps"])
    p = (s["p"] if s["master"] is None else s["master"]).view(-1, BLOCK).float()
    p = p * (1 - ADAM["lr"] * s["decay"]) - update * (ADAM["lr"] / (1 - b1 ** t))
    s["p"].copy_(p.view(-1))
    if s["master"] is not None:
        s["master"].copy_(p.view(-1))
    if eight:
        for name, x in (("m", m), ("v", root)):
            top = x.abs().amax(1, keepdim=True)
            code = torch.where(top < 1e-30, 0.0, x * (448 / top)).to(E4M3)
            if name == "v":  # a root that is not zero keeps the smallest code
                code = torch.where((code.float() == 0) & (x > 0) & (top >= 1e-30), 2.0 ** -9, code.float()).to(E4M3)
            s[name].copy_(code.view(-1))
            s[name + "_scale"].copy_(torch.where(top < 1e-30, 0.0, top / 448)[:, 0])
    else:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
    return _adam_outputs(s)


def work(case):
    op = case["op"]
    if op in ("dispatch", "combine", "combine_backward"):
        T, k, E, H, b = case["T"], case["top_k"], case["E"], case["H"], SIZE[case["dtype"]]
        P = T * k
        if op == "dispatch":
            return {"bytes": T * H * b + P * H * b + 12 * P + 4 * (E + 1), "flops": P}
        if op == "combine":
            return {"bytes": P * H * b + T * H * b + (8 if case["weighted"] else 4) * P, "flops": 2 * P * H}
        return {"bytes": 2 * P * H * b + T * H * b + 16 * P + T * E * (4 if case["norm"] else 8),
                "flops": 3 * P * H + 4 * T * E}
    if op == "embed":
        N, H, b = case["N"], case["H"], SIZE[case["dtype"]]
        return {"bytes": 2 * N * H * b + N * (8 if case["wide_ids"] else 4), "flops": N * H}
    if op == "embed_backward":
        N, V, H = case["N"], case["V"], case["H"]
        return {"bytes": N * H * SIZE[case["dtype"]] + V * H * SIZE[case["table"]] + N * (8 if case["wide_ids"] else 4),
                "flops": N * H}
    if op == "policy_loss":
        N, V, b = case["N"], case["V"], SIZE[case["dtype"]]
        read = N * V * b * (1 - case["masked"])
        return {"bytes": int(read + (N * V * b if case["grad"] else 0) + 32 * N),
                "flops": int(N * (1 - case["masked"]) * V * (8 if case["grad"] else 4))}
    n, b = sum(n for n, _ in _adam_shapes(case)), SIZE[case["dtype"]]
    state = 4 * 4 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": int(n * (b + (b + 8 if case["master"] else 2 * b) + state)), "flops": 16 * n}


# ----------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        k, E = case["top_k"], case["E"]
        e = s["idx"].cpu().numpy().reshape(-1)
        pairs = np.nonzero((e >= 0) & (e < E))[0]
        pairs = pairs[np.lexsort((pairs, e[pairs]))]
        perm = np.full(e.size, -1, np.int32)
        perm[:pairs.size] = pairs
        inv = np.full(e.size, -1, np.int32)
        inv[pairs] = np.arange(pairs.size)
        offsets = np.concatenate([[0], np.cumsum(np.bincount(e[pairs], minlength=E))]).astype(np.int32)
        xs = torch.zeros(e.size, case["H"], dtype=torch.float64, device="cuda")
        xs[:pairs.size] = s["x"][torch.from_numpy(pairs // k).cuda()].double()
        return [offsets, perm, inv, xs]
    if op in ("combine", "combine_backward"):
        T, k = case["T"], case["top_k"]
        inv = s["inv"].view(T, k).long()
        at = [inv[:, j].clamp(min=0) for j in range(k)]
        on = [(inv[:, j] >= 0).double()[:, None] for j in range(k)]
        if op == "combine":
            out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
            for j in range(k):
                wj = s["w"][:, j:j + 1].double() if case["weighted"] else 1.0
                out += on[j] * wj * s["ys"][at[j]].double()
            return [out]
        d, w = s["dout"].double(), s["w"].double()
        dys = torch.zeros(T * k, case["H"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            here = inv[:, j] >= 0
            dys[inv[here, j]] = w[here, j:j + 1] * d[here]
            dw[:, j] = torch.einsum("th,th->t", s["ys"][at[j]].double() * on[j], d)
        prob = torch.softmax(s["logits"].double(), 1)
        chosen = torch.nn.functional.one_hot(s["idx"].long(), case["E"]).double()  # [T, k, E]
        up = torch.einsum("tke,tk->te", chosen, dw)
        if case["norm"]:
            prob = torch.einsum("tke,tk->te", chosen, w)
        return [dys, dw, prob * (up - torch.einsum("tk,tk->t", w, dw)[:, None])]
    if op == "embed":
        return [s["weights"].double()[s["ids"].long()] * s["scale"]]
    if op == "embed_backward":
        ids, order = torch.sort(s["ids"].long())
        run_sum = torch.cumsum(s["dout"][order].double(), 0)
        rows, counts = torch.unique_consecutive(ids, return_counts=True)
        ends = run_sum[torch.cumsum(counts, 0) - 1]
        grad = torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
        grad[rows] = torch.diff(ends, dim=0, prepend=torch.zeros_like(ends[:1])) * s["scale"]
        return [grad]
    if op == "policy_loss":
        N, V = case["N"], case["V"]
        row = torch.zeros(N, dtype=torch.float64, device="cuda")
        logps = torch.zeros_like(row)
        grad = torch.zeros(N, V, dtype=torch.float64, device="cuda") if case["grad"] else None
        for i in range(0, N, 512):
            at = slice(i, min(N, i + 512))
            z, y = s["logits"][at].double(), s["targets"][at]
            w, a = s["weight"][at].double(), s["adv"][at].double()
            use = (w != 0).double()
            lse = torch.logsumexp(z, 1)
            lp = z[torch.arange(len(y), device=y.device), y] - lse
            ratio, back = torch.exp(lp - s["old"][at].double()), torch.exp(s["ref"][at].double() - lp)
            bounded = torch.minimum(torch.maximum(ratio, torch.full_like(ratio, 1 - CLIP_LOW)),
                                    torch.full_like(ratio, 1 + CLIP_HIGH))
            logps[at] = use * lp
            row[at] = use * (KL_COEF * (back - torch.log(back) - 1) - torch.minimum(ratio * a, bounded * a))
            if grad is not None:
                c = w * (KL_COEF * (1 - back) - (ratio * a <= bounded * a).double() * ratio * a)
                grad[at] = -c[:, None] * torch.exp(z - lse[:, None])
                grad[at][torch.arange(len(y), device=y.device), y] += c
        return [(s["weight"].double() * row).sum().view(1), row, logps, grad]
    b1, b2, t = ADAM["beta1"], ADAM["beta2"], ADAM["step"]
    eight = case["bits"] == 8
    grad = s["grad"].double() * float(s["grad_scale"])
    m, second = s["m"].double(), s["v"].double()
    if eight:
        m = (m.view(-1, BLOCK) * s["m_scale"].double()[:, None]).view(-1)
        second = (second.view(-1, BLOCK) * s["v_scale"].double()[:, None]).view(-1) ** 2
    m = b1 * m + (1 - b1) * grad
    second = b2 * second + (1 - b2) * grad ** 2
    old = (s["p"] if s["master"] is None else s["master"]).double()
    new = old - ADAM["lr"] * ((m / (1 - b1 ** t)) / (torch.sqrt(second / (1 - b2 ** t)) + ADAM["eps"]) +
                              s["decay"].double().expand(-1, BLOCK).reshape(-1) * old)
    out = {"p": new}
    if s["master"] is not None:
        out["master"] = new
    if not eight:
        return {**out, "m": m, "v": second}
    for name, x in (("m", m), ("v", torch.sqrt(second))):
        scale = x.view(-1, BLOCK).abs().amax(1) / 448
        code = (x.view(-1, BLOCK) / torch.where(scale > 0, scale, 1.0)[:, None]).to(E4M3).double()
        if name == "v":
            code = torch.where((code == 0) & (x.view(-1, BLOCK) > 0), 2.0 ** -9, code)
        out[name], out[name + "_scale"] = code.view(-1), scale
    return out
