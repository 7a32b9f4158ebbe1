"""Policy-gradient training of a small MoE language model, one token ahead.

    python examples/train_step.py [steps]

Every step runs the training operators around the products: embedding lookup,
routing (ftmoe_route_static), dispatch to the experts, combine, the clipped
policy loss with its KL term, the gradients of all of them, and one AdamW step
over all tensors.  The products themselves are torch matmuls.

The model: x = table[ids] sqrt(H), z = x + sum_j w_j expert_j(x) with SwiGLU
experts, logits = z W_out.  Its task: for token t, choose (7 t + 3) mod V; the
reward of a sampled choice is 1 or 0.
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_mixture_experts_counting_gb300 import ftmoe  # noqa: E402

BF16 = torch.bfloat16


class Model:
    """Weights, gradients, optimiser state (8 or 32 bits) and the buffers of one step."""

    def __init__(self, V=64, H=256, E=16, k=4, I=128, T=512, bits=8, device="cuda", seed=0):
        self.V, self.H, self.E, self.k, self.I, self.T = V, H, E, k, I, T
        self.g = torch.Generator(device=device)
        self.g.manual_seed(seed)
        new = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device=device)
        draw = lambda *s, std: torch.randn(*s, generator=self.g, device=device) * std
        self.master = {"table": draw(V, H, std=1 / math.sqrt(H)), "gate_up": draw(E, H, 2 * I, std=1 / math.sqrt(H)),
                       "down": draw(E, I, H, std=1 / math.sqrt(I)), "out": draw(H, V, std=0.5 / math.sqrt(H))}
        self.p = {n: m.to(BF16) for n, m in self.master.items()}
        self.p["router"] = draw(E, H, std=1 / math.sqrt(H))  # fp32, its own master
        self.grad = {n: torch.zeros_like(v) for n, v in self.p.items()}
        self.grad["table"] = new(V, H, dtype=torch.float32)
        self.ref_out = self.p["out"].clone()  # the reference policy differs in nothing else
        state = []
        for n, v in self.p.items():
            dtype = torch.uint8 if bits == 8 else torch.float32
            t = dict(p=v, g=self.grad[n], master=self.master.get(n), m=torch.zeros_like(v, dtype=dtype),
                     v=torch.zeros_like(v, dtype=dtype), weight_decay=0.0 if n == "router" else 0.01)
            if bits == 8:
                blocks = -(-v.numel() // 256)
                t["m_scale"] = torch.zeros(blocks, device=device)
                t["v_scale"] = torch.zeros(blocks, device=device)
            state.append(t)
        self.tensors = ftmoe.adamw_list(state)
        P = T * k
        i32 = lambda n: new(n, dtype=torch.int32)
        f32 = lambda *s: new(*s, dtype=torch.float32)
        self.x, self.y, self.dx = new(T, H), new(T, H), new(T, H)
        self.xs, self.ys, self.dxs = new(P, H), new(P, H), new(P, H)
        self.idx, self.w, self.dw, self.droute = new(T, k, dtype=torch.int32), f32(T, k), f32(T, k), f32(T, E)
        self.offsets, self.perm, self.inv = i32(E + 1), i32(P), i32(P)
        self.loss, self.row_loss, self.logp, self.dlogits = f32(1), f32(T), f32(T), new(T, V)
        self.workspace = new(ftmoe.ftmoe_embed_workspace(T, H), dtype=torch.uint8)

    def forward(self, ids):
        """Logits [T, V] of the tokens; keeps what the gradient needs."""
        T, H, E, k, p = self.T, self.H, self.E, self.k, self.p
        ftmoe.ftmoe_embed(p["table"], self.V, H, ids, T, math.sqrt(H), self.x)
        ftmoe.ftmoe_route_static(self.x, T, H, p["router"], None, E, k, True, self.idx, self.w, self.offsets, self.perm,
                                 self.inv)
        ftmoe.ftmoe_dispatch(self.x, T, H, self.idx, k, E, self.offsets, self.perm, self.inv, self.xs)
        bounds = self.offsets.tolist()
        self.groups = [(e, slice(bounds[e], bounds[e + 1])) for e in range(E) if bounds[e] < bounds[e + 1]]
        self.gu = torch.empty(T * k, 2 * self.I, dtype=BF16, device=self.x.device)
        for e, s in self.groups:
            torch.matmul(self.xs[s], p["gate_up"][e], out=self.gu[s])
        gate, up = self.gu.float().chunk(2, 1)
        self.h = (torch.nn.functional.silu(gate) * up).to(BF16)
        for e, s in self.groups:
            torch.matmul(self.h[s], p["down"][e], out=self.ys[s])
        ftmoe.ftmoe_combine(self.ys, T, H, k, self.inv, self.w, self.y)
        self.z = self.x + self.y
        return self.z @ p["out"]

    def backward(self, ids):
        """Gradients of every weight from self.dlogits."""
        T, H, E, k, p, grad = self.T, self.H, self.E, self.k, self.p, self.grad
        torch.matmul(self.z.t(), self.dlogits, out=grad["out"])
        dz = self.dlogits @ p["out"].t()
        dys = self.ys  # the experts' outputs are not needed again: their rows become their gradients
        ftmoe.ftmoe_combine_backward(dz, self.ys, T, H, k, self.inv, self.w, dys, self.dw)
        dh = torch.empty_like(self.h)
        for n in ("gate_up", "down"):
            grad[n].zero_()  # an expert without tokens has no gradient
        for e, s in self.groups:
            torch.matmul(self.h[s].t(), dys[s], out=grad["down"][e])
            torch.matmul(dys[s], p["down"][e].t(), out=dh[s])
        gate, up = self.gu.float().chunk(2, 1)
        sig = torch.sigmoid(gate)
        dh = dh.float()
        dgu = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1).to(BF16)
        for e, s in self.groups:
            torch.matmul(self.xs[s].t(), dgu[s], out=grad["gate_up"][e])
            torch.matmul(dgu[s], p["gate_up"][e].t(), out=self.dxs[s])
        ftmoe.ftmoe_combine(self.dxs, T, H, k, self.inv, None, self.dx)  # the dispatch's gradient
        ftmoe.ftmoe_route_backward(None, self.idx, self.w, self.dw, T, E, k, True, self.droute)
        torch.matmul(self.droute.t(), self.x.float(), out=grad["router"])
        dx = (dz.float() + self.dx.float() + self.droute @ p["router"]).to(BF16)
        ftmoe.ftmoe_embed_backward(dx, ids, T, self.V, H, math.sqrt(H), -1, grad["table"], False, self.workspace)

    def step(self, t, lr=3e-3):
        """Sample, reward, learn; returns the mean reward (a device scalar)."""
        dev = self.x.device
        ids = torch.randint(0, self.V, (self.T,), generator=self.g, device=dev)
        logits = self.forward(ids)
        choice = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=self.g)[:, 0]
        reward = (choice == (7 * ids + 3) % self.V).float()
        take = lambda l: torch.log_softmax(l.float(), 1).gather(1, choice[:, None])[:, 0]
        args = ftmoe.policy_args(logits, choice, take(logits), take(self.z @ self.ref_out), (reward - reward.mean()) * 4,
                                 None, self.loss, self.row_loss, self.logp, self.dlogits, kl_coef=0.001)
        ftmoe.ftmoe_policy_loss(args)
        self.backward(ids)
        ftmoe.ftmoe_adamw(self.tensors, lr, 0.9, 0.95, step=t)
        return reward.mean()


def main(steps: int = 200) -> float:
    model = Model()
    reward = 0.0
    for t in range(1, steps + 1):
        reward = model.step(t)
        if t % 25 == 0 or t == 1:
            print(f"step {t}: mean reward {float(reward):.3f}")
    if ftmoe.ftmoe_ops_status():
        raise RuntimeError("a kernel met an index out of range")
    return float(reward)


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
