"""Adapters for many users over a frozen 4-bit channel mixer: serving a mixed batch, and one training step from 8-bit checkpoints.

    n = norm(x),  h = relu(W1 n + b1 + B1_e A1_e n),  out = x + W2 h + b2 + B2_e A2_e h

x is NHWC and each image belongs to a user, whose adapters (A1_e, B1_e, A2_e, B2_e) it goes through; W1 and W2 are the same for all, frozen, with microscaled
4-bit operands.  Training moves the adapters and the norm; between the passes it keeps x, n and h as 8-bit checkpoints, half of what bf16 takes.
The gradient passes through the 4-bit quantisers as if they were not there.

    python examples/adapter_tuning.py [--steps 30] [--images 8] [--size 28] [--channels 64] [--hidden 256] [--rank 8] [--users 3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import split_gemm_gb300 as sg  # noqa: E402


class Frozen:
    """The shared weights in 4 bits, along the sums of the forward and of the backward pass."""

    def __init__(self, channels: int, hidden: int, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        w1 = (torch.randn(hidden, channels, generator=g) * (2 / channels) ** 0.5).to(device)
        w2 = (torch.randn(channels, hidden, generator=g) * (1 / hidden) ** 0.5).to(device)
        self.w1, self.w1_t = sg.mxfp4_quantize(w1), sg.mxfp4_quantize(w1, transpose=True)
        self.w2, self.w2_t = sg.mxfp4_quantize(w2), sg.mxfp4_quantize(w2, transpose=True)
        self.b1, self.b2 = torch.zeros(hidden, device=device), torch.zeros(channels, device=device)


def init(channels: int, hidden: int, rank: int, users: int, seed: int = 0, device="cuda"):
    """What is trained, fp32: adapters that begin as nothing, and the norm."""
    g = torch.Generator().manual_seed(seed)
    down = lambda cols: (torch.randn(users, rank, cols, generator=g) / cols ** 0.5).to(device)  # noqa: E731
    return {"a1": down(channels), "b1": torch.zeros(users, hidden, rank, device=device),
            "a2": down(hidden), "b2": torch.zeros(users, channels, rank, device=device),
            "gamma": torch.ones(channels, device=device), "beta": torch.zeros(channels, device=device)}


def plan_of(users_of_images, x, users: int):
    """The plan of a batch x [N, H, W, C] whose image i belongs to users_of_images[i] (int32; say -1 for none)."""
    n, h, w, _ = x.shape
    return sg.adapter_plan(users_of_images.view(n, 1, 1).expand(n, h, w).contiguous(), users)


def serve(frozen, p, x, plan):
    """The block's output, fp32; x bf16."""
    a1, b1, a2, b2 = (p[k].bfloat16() for k in ("a1", "b1", "a2", "b2"))
    n, _, _ = sg.layer_norm_fwd(x, p["gamma"], p["beta"], out_dtype=torch.bfloat16)
    y1 = sg.mxfp4_matmul(sg.mxfp4_quantize(n), frozen.w1, frozen.b1)
    h, _ = sg.adapter_fwd(y1, n, a1, b1, plan, relu=True, out_dtype=torch.bfloat16)
    y2 = sg.mxfp4_matmul(sg.mxfp4_quantize(h), frozen.w2, frozen.b2)
    sg.adapter_fwd_into(y2, y2, h, a2, b2, plan)
    return x.float() + y2.view(x.shape)


def gradients(frozen, p, x, target, plan):
    """Mean squared error of the block's output, its gradient for each parameter, and for x."""
    channels = x.shape[-1]
    x = x.reshape(-1, channels)
    a1, b1, a2, b2 = (p[k].bfloat16() for k in ("a1", "b1", "a2", "b2"))
    n, mean, rstd = sg.layer_norm_fwd(x, p["gamma"], p["beta"], out_dtype=torch.bfloat16)
    y1 = sg.mxfp4_matmul(sg.mxfp4_quantize(n), frozen.w1, frozen.b1)
    h, m1 = sg.adapter_fwd(y1, n, a1, b1, plan, relu=True, out_dtype=torch.bfloat16)
    y2 = sg.mxfp4_matmul(sg.mxfp4_quantize(h), frozen.w2, frozen.b2)
    y, m2 = sg.adapter_fwd(y2, h, a2, b2, plan)
    err = x.float() + y - target.reshape(-1, channels)
    loss = err.square().mean()
    x8, n8, h8, on = sg.mxint8_quantize(x), sg.mxint8_quantize(n), sg.mxint8_quantize(h), h > 0  # a small h is 0 in h8
    del n, h, y1, y2, y

    dy = err * (2 / err.numel())
    dy16 = dy.bfloat16()
    dh, da2, db2 = sg.adapter_bwd(dy16, h8, m2, a2, b2, plan, dx=sg.mxfp4_matmul(sg.mxfp4_quantize(dy), frozen.w2_t), out_dtype=torch.bfloat16)
    dh = dh * on
    dn, da1, db1 = sg.adapter_bwd(dh, n8, m1, a1, b1, plan, dx=sg.mxfp4_matmul(sg.mxfp4_quantize(dh), frozen.w1_t))
    dx, dgamma, dbeta = sg.mxint8_layer_norm_bwd(dn, x8, mean, rstd, p["gamma"])
    return loss, {"a1": da1, "b1": db1, "a2": da2, "b2": db2, "gamma": dgamma, "beta": dbeta}, dx + dy


def train(frozen, p, x, target, plan, steps: int, rate: float = 0.5):
    """Plain gradient descent; returns the loss of each step."""
    losses = []
    for _ in range(steps):
        loss, grad, _ = gradients(frozen, p, x, target, plan)
        for name, value in grad.items():
            p[name] -= rate * value
        losses.append(loss)
    return torch.stack(losses)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 30), ("images", 8), ("size", 28), ("channels", 64), ("hidden", 256), ("rank", 8), ("users", 3)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    torch.manual_seed(1)
    x = torch.randn(a.images, a.size, a.size, a.channels, device="cuda").bfloat16()
    who = torch.arange(a.images, dtype=torch.int32, device="cuda") % a.users
    target = torch.stack([v.float().roll(int(e) + 1, dims=-1) for v, e in zip(x, who)])  # each user's channels move by another step
    frozen, p, plan = Frozen(a.channels, a.hidden), init(a.channels, a.hidden, a.rank, a.users), plan_of(who, x, a.users)
    losses = train(frozen, p, x, target, plan, a.steps)
    served = serve(frozen, p, x, plan)
    print("loss %.4f -> %.4f in %d steps; served %.4f" % (losses[0], losses[-1], a.steps, (served - target).square().mean()))


if __name__ == "__main__":
    main()
