"""A convolution block with a 4-bit channel mixer: serving and one training step, every operator as it would be used.

    out = x + W2 relu(W1 norm(conv3x3(x)) + b1) + b2

x is NHWC; conv3x3 runs in bf16 (conv2d_fwd), the norm is over the channels, and W1 and W2 are pointwise
convolutions with microscaled 4-bit operands.  Training keeps fp32 weights and quantises both operands of every
product along its own sum, weights and activations afresh in each step; the gradient passes through the quantisers as if they were not there.

    python examples/pointwise_block.py [--steps 30] [--batch 8] [--size 28] [--channels 64] [--hidden 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import split_gemm_gb300 as sg  # noqa: E402


def init(channels: int, hidden: int, seed: int = 0, device="cuda"):
    """The block's fp32 parameters."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *shape, scale: (torch.randn(*shape, generator=g) * scale).to(device)  # noqa: E731
    return {
        "conv": rand(channels, 3, 3, channels, scale=(2 / (9 * channels)) ** 0.5),
        "gamma": torch.ones(channels, device=device), "beta": torch.zeros(channels, device=device),
        "w1": rand(hidden, channels, scale=(2 / channels) ** 0.5), "b1": torch.zeros(hidden, device=device),
        "w2": rand(channels, hidden, scale=0.5 / hidden ** 0.5), "b2": torch.zeros(channels, device=device),
    }


class Serving:
    """The block with its weights quantised once; x is [N, H, W, C] bf16."""

    def __init__(self, p):
        self.conv, self.gamma, self.beta, self.b1, self.b2 = p["conv"].bfloat16(), p["gamma"], p["beta"], p["b1"], p["b2"]
        self.w1, self.w2 = sg.mxfp4_quantize(p["w1"]), sg.mxfp4_quantize(p["w2"])

    def __call__(self, x):
        u = sg.conv2d_fwd(x, self.conv, padding=1)
        a = sg.layer_norm_mxfp4(u, self.gamma, self.beta)
        h = sg.mxfp4_matmul(a, self.w1, self.b1, relu=True, out_dtype=torch.bfloat16)
        y = sg.mxfp4_matmul(sg.mxfp4_quantize(h), self.w2, self.b2)
        return x.float() + y.view(x.shape)


def gradients(p, x, target):
    """Mean squared error of the block's output, and its gradient for each parameter."""
    channels = x.shape[-1]
    # forward, each activation in both forms: by rows for its product, transposed for the weight's gradient
    u = sg.conv2d_fwd(x, p["conv"].bfloat16(), padding=1)
    n, mean, rstd = sg.layer_norm_fwd(u, p["gamma"], p["beta"], out_dtype=torch.bfloat16)
    a, a_t = sg.mxfp4_quantize_both(n)
    h = sg.mxfp4_matmul(a, sg.mxfp4_quantize(p["w1"]), p["b1"], relu=True, out_dtype=torch.bfloat16)
    qh, qh_t = sg.mxfp4_quantize_both(h)
    y = sg.mxfp4_matmul(qh, sg.mxfp4_quantize(p["w2"]), p["b2"])
    err = x.float().view(-1, channels) + y - target.reshape(-1, channels)
    loss = err.square().mean()

    dy = err * (2 / err.numel())
    g, g_t = sg.mxfp4_quantize_both(dy)
    dw2 = sg.mxfp4_matmul(g_t, qh_t)
    dh = sg.mxfp4_matmul(g, sg.mxfp4_quantize(p["w2"], transpose=True)) * (h > 0)
    q, q_t = sg.mxfp4_quantize_both(dh)
    dw1 = sg.mxfp4_matmul(q_t, a_t)
    dn = sg.mxfp4_matmul(q, sg.mxfp4_quantize(p["w1"], transpose=True))
    du, dgamma, dbeta = sg.layer_norm_bwd(dn.view(u.shape), u, mean, rstd, p["gamma"])
    dconv = sg.conv2d_bwd_weight(x, du.bfloat16(), tuple(p["conv"].shape), padding=1)
    return loss, {"conv": dconv, "gamma": dgamma, "beta": dbeta, "w1": dw1, "b1": dh.sum(0), "w2": dw2, "b2": dy.sum(0)}


def train(p, x, target, steps: int, rate: float = 0.5):
    """Plain gradient descent; returns the loss of each step."""
    losses = []
    for _ in range(steps):
        loss, grad = gradients(p, x, target)
        for name, value in grad.items():
            p[name] -= rate * value
        losses.append(loss)
    return torch.stack(losses)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 30), ("batch", 8), ("size", 28), ("channels", 64), ("hidden", 256)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    torch.manual_seed(1)
    x = torch.randn(a.batch, a.size, a.size, a.channels, device="cuda").bfloat16()
    target = x.float().roll(1, dims=2)  # each pixel's left neighbour: the block has to learn it
    p = init(a.channels, a.hidden)
    losses = train(p, x, target, a.steps)
    served = Serving(p)(x)
    print("loss %.4f -> %.4f in %d steps; served %.4f" % (losses[0], losses[-1], a.steps, (served - target).square().mean()))


if __name__ == "__main__":
    main()
