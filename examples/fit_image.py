"""Fits a small image network to one image by SSIM: the loss and the training
operators in one loop.

    python examples/fit_image.py [--steps 300] [--size 256] [--width 512] [--blocks 4] [--attention]

The network maps a learned code for each 16 x 16 patch to its pixels through
blocks of two linear layers.  Between the blocks lies S.block_norm: the block's
output is normed, gated and scaled, added to an fp32 residual stream, and that is
normed for the next block.  With --attention a block is two: attention over the
patches (S.rotary turns queries and keys by their row and column, S.attention), and
a gated feed-forward layer (S.gated_linear).  Weights are bf16 with fp32 masters.  S.loss_and_grad
gives the loss and the image's gradient in one launch; S.AdamW clips and updates.
Nothing in a step waits for the GPU.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ssim_loss_amd as S  # noqa: E402

PATCH = 16
HEAD = 64  # elements of an attention head: half of them turn by the patch's row, half by its column


class Net:
    """Weights are leaves in a list, as the optimizer takes them."""

    def __init__(self, side, width, blocks, seed=0, attention=False):
        if attention and width % HEAD:
            raise ValueError(f"attention needs a width that is a multiple of {HEAD}")
        rng = torch.Generator(device="cuda").manual_seed(seed)
        tokens = (side // PATCH) ** 2
        self.side, self.half, self.full = side, [], []

        def matrix(rows, columns):
            w = torch.randn(rows, columns, generator=rng, device="cuda") * columns ** -0.5
            self.half.append(w.bfloat16().requires_grad_(True))
            return self.half[-1]

        def vector(value):
            self.full.append(torch.full((width,), value, device="cuda", requires_grad=True))
            return self.full[-1]

        self.code = torch.randn(1, tokens, width, generator=rng, device="cuda").requires_grad_(True)
        self.full.append(self.code)
        self.attention = attention
        if attention:
            n = side // PATCH
            at = torch.arange(tokens, device="cuda")
            self.positions = torch.stack([at // n, at % n], 1)
            # for each block: queries, keys and values in one layer, the layer out; the gated layer's two and the one
            # out; scale, post and pre weight of both joints
            self.blocks = [(matrix(3 * width, width), matrix(width, width), matrix(2 * width, width),
                            matrix(2 * width, width), matrix(width, 2 * width),
                            *(vector(v) for v in (0.5, 1.0, 1.0, 0.5, 1.0, 1.0))) for _ in range(blocks)]
        else:
            # for each block: the layers in and out, the gate's layer; scale, post and pre weight
            self.blocks = [(matrix(2 * width, width), matrix(width, 2 * width), matrix(width, width),
                            vector(0.5), vector(1.0), vector(1.0)) for _ in range(blocks)]
        self.head = matrix(3 * PATCH * PATCH, width)

    def parameters(self):
        return self.half + self.full

    def attend(self, stream, h):
        for w_qkv, w_out, w_gate, w_up, w_down, *joints in self.blocks:
            whole = F.linear(h, w_qkv).unflatten(-1, (3, -1, HEAD))  # [1, tokens, 3, heads, HEAD]
            q, k = S.rotary(whole[:, :, 0], whole[:, :, 1], self.positions, (HEAD // 2, HEAD // 2))
            branch = F.linear(S.attention(q, k, whole[:, :, 2]).flatten(2), w_out)
            stream, h = S.block_norm(stream, branch, None, *joints[:3])
            branch = F.linear(S.gated_linear(h, w_gate, w_up), w_down)
            stream, h = S.block_norm(stream, branch, None, *joints[3:])
        return h

    def __call__(self):
        stream, h = self.code, self.code.bfloat16()
        if self.attention:
            return self.image(self.attend(stream, h))
        for w_in, w_out, w_gate, scale, post, pre in self.blocks:
            branch = F.linear(F.gelu(F.linear(h, w_in)), w_out)
            stream, h = S.block_norm(stream, branch, gate=F.linear(h, w_gate), scale=scale,
                                     post_weight=post, pre_weight=pre, gate_act="sigmoid")
        return self.image(h)

    def image(self, h):
        n = self.side // PATCH
        pixels = torch.sigmoid(F.linear(h, self.head).float())
        return pixels.view(n, n, 3, PATCH, PATCH).permute(2, 0, 3, 1, 4).reshape(1, 3, self.side, self.side)


def target_image(side):
    """Smooth colours with rings and a grid of edges, values in [0, 1]."""
    y, x = torch.meshgrid(*[torch.linspace(-1, 1, side, device="cuda")] * 2, indexing="ij")
    r = (x * x + y * y).sqrt()
    rings = 0.5 + 0.25 * torch.sin(20 * r) + 0.25 * torch.sign(torch.sin(9 * x) * torch.sin(7 * y))
    return torch.stack([rings, 0.5 + 0.5 * x * y, 0.5 + 0.5 * torch.cos(5 * r)])[None].clamp(0, 1).contiguous()


def fit(steps=300, size=256, width=512, blocks=4, lr=2e-3, report=None, attention=False):
    """Returns the loss before each step and the gradients' norms, as tensors
    on the GPU."""
    net, target = Net(size, width, blocks, attention=attention), target_image(size)
    parameters = net.parameters()
    optimizer = S.AdamW(parameters, lr=lr, max_norm=1.0, weight_decay=0.0,
                        masters=[p.detach().float() if p.dtype == torch.bfloat16 else None for p in parameters])
    losses, norms = [], []
    for step in range(steps):
        image = net()
        loss, gradient, _ = S.loss_and_grad(image.detach(), target, "valid", grad2=False)
        optimizer.zero_grad()
        image.backward(gradient)
        norms.append(optimizer.step())
        losses.append(loss)
        if report and (step % report == 0 or step == steps - 1):
            print(f"step {step}: loss {float(loss):.4f}, gradient norm {float(norms[-1]):.4f}", flush=True)
    return torch.stack([l.reshape(()) for l in losses]), torch.stack(norms)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--size", type=int, default=256, help=f"side of the image, a multiple of {PATCH}")
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--blocks", type=int, default=4)
    ap.add_argument("--attention", action="store_true", help="blocks of attention and a gated layer")
    a = ap.parse_args()
    if a.size % PATCH or a.size < PATCH:
        ap.error(f"--size must be a multiple of {PATCH}")
    if a.attention and a.width % HEAD:
        ap.error(f"--width must be a multiple of {HEAD} with --attention")
    fit(a.steps, a.size, a.width, a.blocks, report=50, attention=a.attention)
