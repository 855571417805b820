"""A small decoder that predicts Gaussians from images, trained through the rasteriser.

    python -m tile_differentiable_rasterizer_amd.token_decoder [--steps 60] [--experts 4] [--optimizer adamw]

Each token stands for a group of Gaussians; the encoder's states are the 16x16 tiles of the cameras'
images.  One layer, as a feed-forward reconstruction would stack them: queries and keys normed by
head and rotated by position (tokens.norm_rotate), attention of the tokens to the states that show
something (tokens.cross_attention, with a key mask), and a gated feed-forward part whose
activations wait for the backward pass as 8-bit codes (tokens.gated8).  A linear head gives the
Gaussians, raster.Rasterizer the images and their gradients, and gs_adam_q16 the step.  The plain
matrix products are torch's.

With experts, each part of the layer starts with a layer norm (tokens.layer_norm) and the feed-forward part
is a choice of several: a router sends each token to the expert with the largest weight, tokens are sorted by expert,
and their products are made group by group (tokens.group_mm).  With the optimizer "adamw" the step goes over the
parameters as a list of tensors (tokens.adamw: moments in 8 bits, decayed weights), which also writes the bfloat16
copies that the next pass multiplies with.
"""
from __future__ import annotations

import argparse
import math

import numpy as np
import torch

from . import raster, scenes, tokens

TILE = raster.TILE


class Render(torch.autograd.Function):
    """The rasteriser as a differentiable function of degree-0 Gaussians."""

    @staticmethod
    def forward(ctx, means, scales, quats, opacities, sh, cam):
        rz = raster.Rasterizer(means, scales, quats, opacities, sh, 0, pair_capacity=16 * means.shape[0])
        fwd = rz.forward(cam, with_keys=False)
        image = fwd.pop("image")  # an output kept here would keep this frame's buffers from being let go
        ctx.rz, ctx.fwd = rz, fwd
        ctx.save_for_backward(means, scales, quats, opacities, sh)
        return image

    @staticmethod
    @tokens.once
    def backward(ctx, dimage):
        ctx.saved_tensors  # read by the rasteriser again: an error if they were changed since
        g = ctx.rz.backward(ctx.fwd, dimage.contiguous())
        return g["dmeans"], g["dscales"], g["dquats"], g["grad_screen"][:, 5], g["dsh"], None


VECTORS = ("wq", "wk", "norm1", "bias1", "norm2", "bias2", "norm3", "bias3")  # float32 in every pass


class Rounded(torch.autograd.Function):
    """A parameter as the bfloat16 copy that the optimizer's step left of it."""

    @staticmethod
    def forward(ctx, parameter, copy):
        return copy.view_as(copy)

    @staticmethod
    def backward(ctx, d):
        return d.float(), None


class Decoder:
    """One decoder layer and its head; every parameter is a view of one flat float32 tensor, so that one fused Adam
    call updates them all."""

    def __init__(self, n_tokens: int, per_token: int = 16, width: int = 256, heads: int = 4, kv_heads: int = 2, hidden: int = 512,
                 device="cuda", seed: int = 0, experts: int = 0, optimizer: str = "adam_q16"):
        if optimizer not in ("adam_q16", "adamw"):
            raise ValueError("optimizer: adam_q16 or adamw")
        self.experts, self.optimizer = experts, optimizer
        self.n_tokens, self.per_token, self.heads, self.kv_heads = n_tokens, per_token, heads, kv_heads
        self.head_dim = width // heads
        kv = kv_heads * self.head_dim
        shapes = dict(start=(n_tokens, width), states=(TILE * TILE * 3, width), q=(width, width), kv=(width, 2 * kv), out=(width, width),
                      up=(width, 2 * hidden), down=(hidden, width), head=(width, per_token * 14), wq=(self.head_dim,), wk=(self.head_dim,))
        if experts:
            shapes.update(up=(experts, width, 2 * hidden), down=(experts, hidden, width), router=(width, experts),
                          norm1=(width,), bias1=(width,), norm2=(width,), bias2=(width,), norm3=(width,), bias3=(width,))
        n = sum(-(-math.prod(s) // 64) * 64 for s in shapes.values())  # each starts on 256 bytes
        self.flat = torch.zeros(n, device=device)
        self.grad = torch.zeros(n, device=device)
        if optimizer == "adam_q16":
            self.adam, self.bounds = raster.adam_state(n, device)
        self.steps, self.p, at = 0, {}, 0
        g = torch.Generator(device=device).manual_seed(seed)
        for name, shape in shapes.items():
            m = math.prod(shape)
            view = self.flat[at: at + m].view(shape)
            if name.startswith("bias"):
                pass
            elif name in VECTORS:
                view.fill_(1.0)
            else:
                view.copy_(torch.randn(shape, generator=g, device=device) * (0.2 if name == "head" else 1.0) / math.sqrt(1 if name == "start" else shape[-2]))
            leaf = view.detach().requires_grad_()
            leaf.grad = self.grad[at: at + m].view(shape)
            self.p[name], at = leaf, at + -(-m // 64) * 64
        if optimizer == "adamw":
            self.state = tokens.adamw_state(list(self.p.values()), bits=8)
            # what the products multiply with: kept up to date by the step; a vector has none
            self.copies = {k: None if k in VECTORS else torch.empty_like(v, dtype=torch.bfloat16) for k, v in self.p.items()}
            self.copied = {}
        # each group's home, on a grid around the origin: the head moves its Gaussians from there
        side = math.ceil(n_tokens ** (1 / 3))
        i = torch.arange(n_tokens, device=device)
        grid = torch.stack([i % side, i // side % side, i // side**2], 1).float()
        self.home = ((grid + 0.5) / side - 0.5).mul(2.4).repeat_interleave(per_token, 0)

    def rotation(self, n: int):
        half = self.head_dim // 2
        angle = torch.arange(n, device=self.flat.device, dtype=torch.float64)[:, None] * 1e4 ** (
            -torch.arange(half, device=self.flat.device, dtype=torch.float64) / half)
        return angle.cos().float(), angle.sin().float()

    def __call__(self, images: torch.Tensor):
        """Gaussians (means, scales, quats, opacities, sh) from images [views, 3, H, W], H and W multiples of 16."""
        if self.optimizer == "adamw":
            for k, v in self.p.items():
                if k not in VECTORS and self.copied.get(k) != v._version:  # changed by something else than the step
                    self.copies[k].copy_(v.detach())
                    self.copied[k] = v._version
            p = {k: v if k in VECTORS else Rounded.apply(v, self.copies[k]) for k, v in self.p.items()}
        else:
            p = {k: v.to(torch.bfloat16) if k not in VECTORS else v for k, v in self.p.items()}
        V, _, H, W = images.shape
        tiles = images.view(V, 3, H // TILE, TILE, W // TILE, TILE).permute(0, 2, 4, 1, 3, 5).reshape(1, -1, 3 * TILE * TILE)
        shown = (tiles.amax(-1) > 0.02).to(torch.uint8)  # tiles of background carry nothing
        states = tiles.to(torch.bfloat16) @ p["states"]
        L, hd = states.shape[1], self.head_dim
        x = p["start"][None]
        norm = lambda x, i: tokens.layer_norm(x, p[f"norm{i}"], p[f"bias{i}"]) if self.experts else x  # noqa: E731
        q = (norm(x, 1) @ p["q"]).view(1, self.n_tokens, self.heads, hd)
        kv = (states @ p["kv"]).view(1, L, 2, self.kv_heads, hd)
        cos, sin = self.rotation(max(L, self.n_tokens))
        q, k = tokens.norm_rotate(q, kv[:, :, 0], p["wq"], p["wk"], cos, sin)
        a = tokens.cross_attention(q, k, kv[:, :, 1], key_mask=shown)
        x = x + a.view(1, self.n_tokens, -1) @ p["out"]
        x = x + self.feed_forward(norm(x, 2), p)
        g = (norm(x, 3) @ p["head"]).float().view(-1, 14)
        means = self.home + 0.5 * torch.tanh(g[:, 0:3])
        scales = torch.exp(-2.3 + torch.tanh(g[:, 3:6]))
        quats = torch.cat([1.0 + g[:, 6:7], g[:, 7:10]], 1)
        opacities = torch.sigmoid(g[:, 10])
        return means, scales.contiguous(), quats, opacities, g[:, 11:14].reshape(-1, 1, 3).contiguous()

    def feed_forward(self, x, p):
        if not self.experts:
            return tokens.gated8(x @ p["up"]) @ p["down"]
        flat = x.view(-1, x.shape[-1])
        weight, expert = torch.softmax((flat @ p["router"]).float(), -1).max(-1)
        # tokens sorted by expert, and where each expert's start
        order = expert.argsort(stable=True)
        offsets = torch.searchsorted(expert[order], torch.arange(self.experts + 1, device=x.device)).int()
        y = tokens.group_mm(tokens.gated8(tokens.group_mm(flat[order], p["up"], offsets)), p["down"], offsets)
        return (torch.zeros_like(y).index_copy(0, order, y) * weight[:, None].to(y.dtype)).view_as(x)

    def step(self, lr: float):
        self.steps += 1
        if self.optimizer == "adamw":
            tokens.adamw(list(self.p.values()), [v.grad for v in self.p.values()], self.state, lr, self.steps, copies=list(self.copies.values()),
                         weight_decay=[0.0 if k in VECTORS or k == "start" else 0.01 for k in self.p])
            self.copied = {k: v._version for k, v in self.p.items()}
            self.grad.zero_()
            return
        raster.adam_q16(self.flat, self.grad, self.adam, self.bounds, lr=lr, step=self.steps)
        self.grad.zero_()


def scene_images(n: int, size: int, views: int):
    """Images [views, 3, size, size] of a synthetic scene and the cameras they are seen from."""
    scene = scenes.sphere_scene(7, n, False)
    cams = [scenes.orbit_camera(2 * math.pi * i / views, size, size, f=size * 0.9) for i in range(views)]
    rz = raster.Rasterizer(*raster.scene_to_device(scene), scene.sh_degree)
    return torch.stack([rz.forward(c)["image"].clone() for c in cams]), cams


def train(steps: int = 60, size: int = 128, views: int = 4, n_tokens: int = 125, lr: float = 2e-3, say=print, experts: int = 0,
          optimizer: str = "adam_q16") -> list:
    """The mean squared errors of the steps."""
    images, cams = scene_images(4000, size, views)
    model = Decoder(n_tokens, experts=experts, optimizer=optimizer)
    losses = []
    for i in range(steps):
        gaussians = model(images)
        loss = sum((Render.apply(*gaussians, cam) - image).square().mean() for cam, image in zip(cams, images)) / views
        loss.backward()
        model.step(lr)
        losses.append(loss.detach())
        if say and (i % 10 == 0 or i == steps - 1):
            say(f"step {i:4d}  mse {losses[-1].item():.5f}", flush=True)
    return [float(x) for x in torch.stack(losses).cpu().numpy().astype(np.float64)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--experts", type=int, default=0, help="experts of the feed-forward part (0: one feed-forward part, no layer norms)")
    ap.add_argument("--optimizer", default="adam_q16", choices=("adam_q16", "adamw"))
    a = ap.parse_args()
    train(a.steps, experts=a.experts, optimizer=a.optimizer)
