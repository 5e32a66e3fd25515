"""Residual layers whose products run in MXFP4, trained and then served.

    python examples/mx_layer.py [--tokens 4096] [--hidden 4096] [--layers 2] [--steps 4]

A layer is x + W norm(x) + b.  In training the weight stays in bf16 and is
quantized for every step; the backward pass quantizes what each of its products
sums over.  For serving the weights are quantized once and the same layer takes
prompts and single tokens: the script decodes a few tokens and checks them
against the pass over all of them.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import blockwise_bit_codebook_amd as kb  # noqa: E402


class NormLinear(torch.autograd.Function):
    """Layer norm and the linear layer behind it, of rows x [tokens, hidden]."""

    @staticmethod
    def forward(ctx, x, norm_weight, norm_bias, weight, bias, eps):
        y = kb.layer_norm(x, norm_weight, norm_bias, eps)
        ctx.save_for_backward(x, y, norm_weight, weight)
        ctx.eps = eps
        return kb.linear_mxfp4_dynamic(y, *kb.quantize_mxfp4(weight), bias=bias)

    @staticmethod
    def backward(ctx, dout):
        x, y, norm_weight, weight = ctx.saved_tensors
        dy, dweight, dbias = kb.linear_mxfp4_backward(dout.contiguous(), y, weight)
        dx, dnorm_weight, dnorm_bias = kb.layer_norm_backward(dy, x, norm_weight, ctx.eps, dx=dy)
        return (dx, dnorm_weight.to(norm_weight.dtype), dnorm_bias.to(norm_weight.dtype), dweight.to(weight.dtype),
                dbias.to(weight.dtype), None)


class MxLayer(torch.nn.Module):
    """x + W norm(x) + b."""

    def __init__(self, hidden, eps=1e-5, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.eps = eps
        self.norm_weight = torch.nn.Parameter(torch.ones(hidden, device=device))
        self.norm_bias = torch.nn.Parameter(torch.zeros(hidden, device=device))
        self.weight = torch.nn.Parameter((torch.randn(hidden, hidden, device=device) * hidden ** -0.5).to(dtype))
        self.bias = torch.nn.Parameter(torch.zeros(hidden, device=device, dtype=dtype))
        self.codes = self.scales = None

    def forward(self, x):
        return x + NormLinear.apply(x, self.norm_weight, self.norm_bias, self.weight, self.bias, self.eps)

    def freeze(self):
        """Quantizes the weight for serve()."""
        self.codes, self.scales = kb.quantize_mxfp4(self.weight.detach())
        return self

    @torch.no_grad()
    def serve(self, x):
        y = kb.layer_norm(x, self.norm_weight, self.norm_bias, self.eps)
        return x + kb.linear_mxfp4_dynamic(y, self.codes, self.scales, bias=self.bias)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--lr", type=float, default=1e-3)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    net = torch.nn.Sequential(*(MxLayer(a.hidden) for _ in range(a.layers)))
    x = torch.randn(a.tokens, a.hidden, device="cuda", dtype=torch.bfloat16)
    target = torch.roll(x, 1, 1)
    opt = torch.optim.SGD(net.parameters(), lr=a.lr)
    for step in range(a.steps):
        torch.cuda.synchronize()
        start = time.perf_counter()
        opt.zero_grad()
        loss = torch.nn.functional.mse_loss(net(x).float(), target.float())
        loss.backward()
        opt.step()
        torch.cuda.synchronize()
        print(f"step {step}: loss {loss.item():.4f}, {(time.perf_counter() - start) * 1e3:.2f} ms")

    layers = [layer.freeze() for layer in net]

    def serve(rows):
        for layer in layers:
            rows = layer.serve(rows)
        return rows
    whole = serve(x)
    tokens = min(4, a.tokens)
    start = time.perf_counter()
    alone = torch.cat([serve(x[i:i + 1]) for i in range(tokens)])
    torch.cuda.synchronize()
    print(f"{tokens} tokens one at a time: {(time.perf_counter() - start) / tokens * 1e6:.0f} us a token")
    # the same codes summed in another order: a bf16 step of a layer's output may
    # move a value to the next code, 1 in 4 of its block's largest at most, in the next layer
    off = (alone.float() - whole[:tokens].float()).abs().max().item()
    print(f"one at a time against all at once: {off:.3g} apart at most")
    return net, x, alone, whole[:tokens]


if __name__ == "__main__":
    main()
