"""Train one top-k MoE layer to imitate another, on one GPU.

Runs the training calls together as a program would: the forward pass in its
steps, the gradient of the combine, of the experts and of the dispatch, the
gate's gradient, clipping by the gradient's norm without a host round trip,
and one AdamW step over all tensors, with moments in 32 or 8 bits:

  python examples/train_layer.py [--steps 60] [--bits 8] [--act swiglu]

The parameters live in fp32; the layer computes with the bf16 copies that the
AdamW step writes.  The gate is E outputs wide, so its gradient is a few torch
operations on [T, E]: with w the renormalised softmax of the chosen scores,
  dlogits[t, ids_j] = w_j (dw_j - sum_i w_i dw_i).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mixture_experts_topk_gb300 as moe  # noqa: E402


def buffer(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Layer:
    """A layer's bf16 weights, and the buffers of a training step of T tokens."""

    def __init__(self, T, H, E, K, F, act="gelu", seed=0):
        self.T, self.H, self.E, self.K, self.F, g = T, H, E, K, F, 2 if act == "swiglu" else 1
        flags = moe.MOE_FLAG_SWIGLU if act == "swiglu" else 0
        self.desc = moe.make_desc(T, H, E, K, F, flags=flags)
        self.ws, self.bws = moe.workspace(self.desc), moe.backward_workspace(self.desc)
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def xavier(*shape):
            bound = (6.0 / (shape[-1] + shape[-2])) ** 0.5
            return buffer(*shape, dtype=torch.float32).uniform_(-bound, bound, generator=gen)

        self.master = {"Wg": xavier(E, H), "W1": xavier(E, g * F, H), "W2": xavier(E, H, F),
                       "b1": torch.zeros(E, g * F, device="cuda"), "b2": torch.zeros(E, H, device="cuda")}
        self.copy = {k: self.master[k].to(torch.bfloat16) for k in ("Wg", "W1", "W2")}
        self.grad = {k: torch.empty_like(self.copy.get(k, v)) for k, v in self.master.items()}
        self.grad["Wg"] = torch.empty_like(self.master["Wg"])
        R = moe.moe_max_rows(self.desc)
        i32 = torch.int32
        self.logits, self.ids, self.w = buffer(T, E, dtype=torch.float32), buffer(T, K, dtype=i32), buffer(T, K, dtype=torch.float32)
        self.count, self.offs, self.src, self.pos = (buffer(n, dtype=i32) for n in (E, E + 1, R, T * K))
        self.x_perm, self.h_perm, self.y_perm = buffer(R, H), buffer(R, F), buffer(R, H)
        self.dy_perm, self.dx_perm, self.dw = buffer(R, H), buffer(R, H), buffer(T, K, dtype=torch.float32)

    def forward(self, x):
        d, c, m, out = self.desc, self.copy, self.master, torch.empty_like(x)
        moe.moe_router_topk(d, x, c["Wg"], None, self.logits, self.ids, self.w, None, self.ws)
        moe.moe_dispatch(d, self.ids, x, self.count, self.offs, self.src, self.pos, self.x_perm, None, self.ws)
        moe.moe_expert_ffn(d, self.x_perm, self.offs, c["W1"], m["b1"], c["W2"], m["b2"], self.h_perm, self.y_perm, self.ws)
        moe.moe_combine(d, self.y_perm, self.pos, self.w, out)
        return out

    def backward(self, x, dout):
        """The parameters' gradients into ``self.grad``; returns x's."""
        d, c, g = self.desc, self.copy, self.grad
        moe.moe_combine_backward(d, dout, self.y_perm, self.pos, self.w, self.dy_perm, self.dw)
        moe.moe_expert_ffn_backward(d, self.x_perm, self.h_perm, self.dy_perm, self.offs, c["W1"], self.master["b1"],
                                    c["W2"], self.dx_perm, g["W1"], g["b1"], g["W2"], g["b2"], self.bws)
        dl = torch.zeros_like(self.logits)
        dl.scatter_(1, self.ids.long(), self.w * (self.dw - (self.w * self.dw).sum(1, keepdim=True)))
        torch.mm(dl.T, x.float(), out=g["Wg"])
        dx = (dl @ c["Wg"].float()).to(x.dtype)
        moe.moe_dispatch_backward(d, self.dx_perm, self.pos, dx, dx)     # onto the gate's part
        return dx


class AdamW:
    """AdamW over a layer's parameters, one plan for each gradient type."""

    def __init__(self, layer, bits=32, weight_decay=0.01):
        def state(v):
            if bits == 32:
                return {"m": torch.zeros_like(v), "v": torch.zeros_like(v)}
            blocks = -(-v.numel() // moe.MOE_ADAMW_BLOCK)
            code = [torch.zeros_like(v, dtype=torch.float8_e4m3fn) for _ in range(2)]
            scale = [torch.zeros(blocks, device="cuda") for _ in range(2)]
            return {"m": code[0], "v": code[1], "m_scale": scale[0], "v_scale": scale[1]}

        tensors = {k: {"p": v, "g": layer.grad[k], "p16": layer.copy.get(k), **state(v),
                       "weight_decay": weight_decay if k in ("W1", "W2") else 0.0} for k, v in layer.master.items()}
        self.plans = [moe.adamw_tensors([t for t in tensors.values() if t["g"].dtype == dt])
                      for dt in (torch.float32, torch.bfloat16)]
        self.grads, self.t = list(layer.grad.values()), 0

    def step(self, lr, clip=1.0):
        norm = torch.stack([g.float().square().sum() for g in self.grads]).sum().sqrt()
        scale = (clip / norm).clamp(max=1.0).reshape(1)
        skip = (~torch.isfinite(norm)).to(torch.int32).reshape(1)        # a bad gradient changes nothing
        self.t += 1
        params = moe.make_adamw(lr=lr, beta2=0.95, step=self.t)
        for plan in self.plans:
            moe.moe_adamw_step(plan, params, scale, skip)


def train(steps=60, T=512, H=256, E=8, K=2, F=512, act="gelu", bits=32, lr=3e-3, log=print):
    """Returns the loss before the first and after the last step."""
    teacher, student = Layer(T, H, E, K, F, act, seed=1), Layer(T, H, E, K, F, act, seed=2)
    optimiser = AdamW(student, bits)
    gen = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for i in range(steps + 1):
        x = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
        target, out = teacher.forward(x), student.forward(x)
        diff = out.float() - target.float()
        losses.append(diff.square().mean())
        if i % 20 == 0:
            log(f"step {i:4d}  loss {losses[-1].item():.5f}")
        if i == steps:
            break
        student.backward(x, (2.0 / T * diff).to(torch.bfloat16))
        optimiser.step(lr)
    if moe.moe_get_device_error(student.bws) != moe.MOE_OK:
        raise RuntimeError("device error flag set")
    return losses[0].item(), losses[-1].item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, default=32, choices=(8, 32))
    ap.add_argument("--act", default="gelu", choices=("gelu", "swiglu"))
    a = ap.parse_args()
    first, last = train(a.steps, act=a.act, bits=a.bits)
    print(f"loss {first:.5f} -> {last:.5f}")
