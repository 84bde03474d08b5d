"""A pre-norm block around the SwiGLU MLP step, trained and then served.

Training: a stack of blocks y = x + MLP(norm(x)) (swiglu_prenorm_mlp) fits a
fixed random map; the gradients of every block are clipped together
(swiglu_clip_grad_norm) before a step of gradient descent with fp32 master
weights.  Serving: the last block's MLP becomes the start of a few experts, and
a handful of tokens runs through norm, router and experts (swiglu_layer_norm,
swiglu_moe_few_layer), one step after another, as a decoder would.

    python examples/prenorm_block.py [--dim 1024] [--inner 2816] [--tokens 2048] [--steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_gemm_epilogue_amd as sw  # noqa: E402


def make_block(D, I, generator):
    """(norm weight, norm bias, W1, W_down): fp32 norm, bf16 matrices"""
    r = lambda *s: torch.randn(*s, generator=generator, device="cuda")  # noqa: E731
    return [torch.ones(D, device="cuda"), torch.zeros(D, device="cuda"), (r(D, 2 * I) * D ** -0.5).bfloat16(),
            (r(I, D) * I ** -0.5).bfloat16()]


def forward(x, blocks):
    for weight, bias, W1, W_down in blocks:
        x = sw.swiglu_prenorm_mlp(x, weight, bias, W1, W_down)
    return x


def train(D=1024, I=2816, tokens=2048, layers=2, steps=30, lr=2.0, max_norm=0.1, seed=0, say=print):
    """Returns (blocks, losses, gradient norms)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [make_block(D, I, g) for _ in range(layers)]
    target_blocks = [make_block(D, I, g) for _ in range(layers)]
    params = [p.requires_grad_() for b in blocks for p in b]
    master = [p.detach().float() for p in params]
    x = torch.randn(tokens, D, generator=g, device="cuda").bfloat16()
    with torch.no_grad():
        want = forward(x, target_blocks).float()
    losses, norms = [], []
    for step in range(steps):
        loss = (forward(x, blocks).float() - want).square().mean()
        loss.backward()
        grads = [p.grad for p in params]
        norm = sw.swiglu_clip_grad_norm(grads, max_norm)
        with torch.no_grad():
            for p, m, d in zip(params, master, grads):
                m -= lr * d.float()
                p.copy_(m)
                p.grad = None
        losses.append(loss.detach())
        norms.append(norm)
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step:3d}  loss {float(losses[-1]):.4f}  gradient norm {float(norm):.4f}")
    return blocks, [float(v) for v in losses], [float(v) for v in norms]


@torch.no_grad()
def serve(block, experts=8, k=2, tokens=4, steps=8, seed=1, say=print):
    """Decode steps x <- x + experts(norm(x)); returns the last x and how often
    each expert was chosen."""
    weight, bias, W1, W_down = block
    D = W1.shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # every expert starts from the trained MLP and differs from it a little
    W1s = torch.stack([W1.float() + 0.1 * r(*W1.shape) * D ** -0.5 for _ in range(experts)]).bfloat16()
    W2s = torch.stack([W_down] * experts).contiguous()
    router = (r(D, experts) * D ** -0.5).bfloat16()
    x = r(tokens, D).bfloat16()
    used = torch.zeros(experts, dtype=torch.int64, device="cuda")
    for _ in range(steps):
        y, ids, _ = sw.swiglu_moe_few_layer(sw.swiglu_layer_norm(x, weight, bias), router, W1s, W2s, k)
        x = x + y
        used += torch.bincount(ids.flatten().long(), minlength=experts)
    say(f"served {tokens} tokens for {steps} steps; experts chosen {used.tolist()}")
    return x, used


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=2816)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    blocks, _, _ = train(a.dim, a.inner, a.tokens, a.layers, a.steps)
    serve([p.detach() for p in blocks[-1]])


if __name__ == "__main__":
    main()
