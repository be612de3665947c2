"""A small transformer that predicts Gaussians from an image, trained through the rasterizer.

The image is cut into 16 x 16 tiles, a token each.  Blocks of attention and a perceptron mix
the tokens; a linear head gives every token a few Gaussians in front of its tile (an offset
inside the tile, depth, scales, quaternion, opacity, colour).  The rasterizer draws them, the
L1 + SSIM loss compares the picture with the image, and the gradients run back through
gs_rasterize_bwd and gs_project_bwd into the network.

The token operators of the package do the hot parts of a block, forward and backward:

    packed projection -> gs_qk_norm_rope -> gs_attention_fwd -> projection -> gs_dropout_add

The plain torch parts are the matrix products, the layer norms and the optimizer.

    python examples/predict_gaussians.py [--steps 200] [--size 128]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch
from torch import nn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import differentiable_gaussian_splatting_gb300 as gs  # noqa: E402
import synthetic_scenes as ss  # noqa: E402

TILE = gs.TILE
RAW = 14  # raw parameters of a Gaussian: offset 2, depth 1, log-scales 3, quaternion 4, logit 1, colour 3


def _workspace(n_bytes: int) -> torch.Tensor:
    return torch.empty(n_bytes, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------
# the package's calls as differentiable functions
# ---------------------------------------------------------------------------
class HeadAttention(torch.autograd.Function):
    """Head norms, rotation and attention on a packed projection [tokens, heads_q + 2 heads_k,
    head_dim] of queries, keys and values; its gradient is written into one packed array."""

    @staticmethod
    def forward(ctx, qkv, q_weight, k_weight, table, heads_k, cu):
        T, heads, D = qkv.shape
        hq = heads - 2 * heads_k
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads_k], qkv[:, hq + heads_k:]
        qn, kn = torch.empty((T, hq, D), dtype=qkv.dtype, device=qkv.device), torch.empty(
            (T, heads_k, D), dtype=qkv.dtype, device=qkv.device)
        gs.gs_qk_norm_rope(q, k, q_weight, k_weight, table, None, qn, kn)
        out, lse = torch.empty_like(qn), torch.empty((hq, T), device=qkv.device)
        batch = 1 if cu is None else cu.numel() - 1
        ws = _workspace(gs.gs_attention_workspace_bytes(T, T, batch, hq, heads_k, D))
        gs.gs_attention_fwd(qn, kn, v, out, lse, ws, cu_q=cu, cu_k=cu)
        ctx.save_for_backward(qkv, q_weight, k_weight, table, qn, kn, out, lse, cu)
        ctx.heads = hq, heads_k
        return out

    @staticmethod
    def backward(ctx, dout):
        qkv, q_weight, k_weight, table, qn, kn, out, lse, cu = ctx.saved_tensors
        hq, hk = ctx.heads
        T, _, D = qkv.shape
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        dqkv = torch.empty_like(qkv)
        dqn, dkn = torch.empty_like(qn), torch.empty_like(kn)
        batch = 1 if cu is None else cu.numel() - 1
        ws = _workspace(gs.gs_attention_workspace_bytes(T, T, batch, hq, hk, D))
        gs.gs_attention_bwd(qn, kn, v, out, lse, dout.contiguous(), dqn, dkn, dqkv[:, hq + hk:], ws,
                            cu_q=cu, cu_k=cu)
        dqw, dkw = torch.empty_like(q_weight), torch.empty_like(k_weight)
        ws = _workspace(gs.gs_qk_norm_rope_workspace_bytes(T, hq, hk, D))
        gs.gs_qk_norm_rope_bwd(q, k, q_weight, k_weight, table, None, dqn, dkn, dqkv[:, :hq],
                               dqkv[:, hq:hq + hk], dqw, dkw, ws)
        return dqkv, dqw, dkw, None, None, None


class DropoutAdd(torch.autograd.Function):
    """residual + dropout(x); rng is the call's own (seed, offset) on the device."""

    @staticmethod
    def forward(ctx, x, residual, rng, p):
        out = torch.empty_like(x)
        gs.gs_dropout_add(x, residual, out, rng, p)
        ctx.rng, ctx.p = rng.clone(), p  # the caller may move rng on before the backward
        return out

    @staticmethod
    def backward(ctx, dout):
        dout = dout.contiguous()
        dx = torch.empty_like(dout)
        gs.gs_dropout_add_bwd(dout, dx, ctx.rng, ctx.p)
        return dx, dout, None, None


class RenderLoss(torch.autograd.Function):
    """The L1 + SSIM loss of the rendered Gaussians against a target image."""

    @staticmethod
    def forward(ctx, means, scales, quats, opacities, sh, raster, target, ws):
        image, _ = raster.forward(means, scales, quats, opacities, sh)
        H, W = image.shape[:2]
        dimage, loss = torch.empty_like(image), torch.empty(4, device=image.device)
        gs.gs_loss_l1_ssim(W, H, image, target, dimage, loss, ws)
        ctx.raster = raster
        ctx.save_for_backward(dimage)
        return loss[0].clone()

    @staticmethod
    def backward(ctx, dloss):
        (dimage,) = ctx.saved_tensors
        g = ctx.raster.backward(dimage * dloss)
        return g.means, g.scales, g.quats, g.opacities, g.sh, None, None, None


# ---------------------------------------------------------------------------
# the network
# ---------------------------------------------------------------------------
def axial_table(rows: int, cols: int, rot: int) -> torch.Tensor:
    """cos | sin [rows * cols, rot] of the tiles of a grid: half of a head's pairs turn with the
    tile's row, half with its column."""
    pairs = rot // 2
    of_row = (pairs + 1) // 2
    i = torch.arange(rows * cols, dtype=torch.float64)
    row, col = torch.div(i, cols, rounding_mode="floor"), i % cols
    f = lambda n: 100.0 ** (-torch.arange(n, dtype=torch.float64) / max(1, n))
    angle = torch.cat([row[:, None] * f(of_row), col[:, None] * f(pairs - of_row)], 1)
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


class Block(nn.Module):
    def __init__(self, width: int, heads: int, heads_k: int, p: float):
        super().__init__()
        self.heads, self.heads_k, self.dim, self.p = heads, heads_k, width // heads, p
        self.norm1, self.norm2 = nn.LayerNorm(width), nn.LayerNorm(width)
        self.qkv = nn.Linear(width, (heads + 2 * heads_k) * self.dim, bias=False)
        self.proj = nn.Linear(width, width, bias=False)
        self.up, self.down = nn.Linear(width, 4 * width), nn.Linear(4 * width, width)
        self.q_weight = nn.Parameter(torch.ones(self.dim))
        self.k_weight = nn.Parameter(torch.ones(self.dim))

    def forward(self, x, table, rng, cu):
        """x [tokens, width] bfloat16; rng [2, 2]: a generator state for each residual branch"""
        lin = lambda m, v: nn.functional.linear(v, m.weight.bfloat16(),
                                                None if m.bias is None else m.bias.bfloat16())
        norm = lambda m, v: nn.functional.layer_norm(v.float(), m.normalized_shape, m.weight,
                                                     m.bias).bfloat16()
        T = x.shape[0]
        qkv = lin(self.qkv, norm(self.norm1, x)).view(T, -1, self.dim)
        y = HeadAttention.apply(qkv, self.q_weight, self.k_weight, table, self.heads_k, cu)
        p = self.p if self.training else 0.0
        x = DropoutAdd.apply(lin(self.proj, y.reshape(T, -1)), x, rng[0], p)
        y = lin(self.down, nn.functional.gelu(lin(self.up, norm(self.norm2, x))))
        return DropoutAdd.apply(y, x, rng[1], p)


class TilePredictor(nn.Module):
    """Gaussians for every 16 x 16 tile of an image (whose sides are multiples of 16)."""

    def __init__(self, rows: int, cols: int, width=256, heads=4, heads_k=2, blocks=3,
                 per_tile=8, p=0.05, seed=0):
        super().__init__()
        torch.manual_seed(seed)
        self.rows, self.cols, self.per_tile = rows, cols, per_tile
        self.embed = nn.Linear(3 * TILE * TILE, width)
        self.blocks = nn.ModuleList([Block(width, heads, heads_k, p) for _ in range(blocks)])
        self.norm = nn.LayerNorm(width)
        self.head = nn.Linear(width, per_tile * RAW)
        nn.init.normal_(self.head.weight, std=0.02)
        # start: spread over the tile, a third of its width across, half opaque, grey
        with torch.no_grad():
            bias = torch.zeros(per_tile, RAW)
            bias[:, :2] = torch.randn(per_tile, 2)
            bias[:, 3:6] = math.log(TILE / 3.0)
            bias[:, 6] = 1.0
            bias[:, 11:14] = 0.5
            self.head.bias.copy_(bias.reshape(-1))
        self.register_buffer("rng", torch.tensor([[seed, i] for i in range(2 * blocks)],
                                                 dtype=torch.int64), persistent=False)
        self.register_buffer("table", axial_table(rows, cols, width // heads), persistent=False)
        self.cuda()

    def tokens(self, image):
        """[tiles, 768] bfloat16 from an image [H, W, 3]"""
        r, c = self.rows, self.cols
        x = image.view(r, TILE, c, TILE, 3).transpose(1, 2).reshape(r * c, -1)
        return nn.functional.linear(x, self.embed.weight, self.embed.bias).bfloat16()

    def forward(self, image, cam):
        """(means, scales, quats, opacities, sh) of all Gaussians, in front of the camera"""
        x = self.tokens(image)
        for i, block in enumerate(self.blocks):
            x = block(x, self.table, self.rng[2 * i:2 * i + 2], None)
        if self.training:
            self.rng[:, 1] += 2 * len(self.blocks)  # the next step's masks
        x = nn.functional.layer_norm(x.float(), self.norm.normalized_shape, self.norm.weight,
                                     self.norm.bias)
        raw = self.head(x).view(self.rows, self.cols, self.per_tile, RAW)
        z = 4.0 + torch.tanh(raw[..., 2])
        at = torch.arange(max(self.rows, self.cols), device="cuda", dtype=torch.float32)
        px = TILE * (at[:self.cols, None] + 0.5 + torch.tanh(raw[..., 0]))
        py = TILE * (at[:self.rows, None, None] + 0.5 + torch.tanh(raw[..., 1]))
        means = torch.stack([(px - cam.cx) / cam.fx * z, (py - cam.cy) / cam.fy * z, z], -1)
        scales = torch.exp(raw[..., 3:6].clamp(-4.0, 4.0)) * (z / cam.fx)[..., None]
        n = self.rows * self.cols * self.per_tile
        sh = raw[..., 11:14] / 0.28209479177387814  # the constant basis function
        return (means.reshape(n, 3).contiguous(), scales.reshape(n, 3).contiguous(),
                raw[..., 6:10].reshape(n, 4).contiguous(),
                torch.sigmoid(raw[..., 10]).reshape(n).contiguous(),
                sh.reshape(n, 1, 3).contiguous())


def target_image(size: int, seed: int = 0) -> torch.Tensor:
    _, y = ss.image_pair(np.random.default_rng(seed), size, size)
    return torch.from_numpy(y).cuda()


def train(steps=200, size=128, lr=3e-4, p=0.05, seed=0, log=None):
    """Fits the predictor to one synthetic image; returns the losses."""
    tiles = size // TILE
    target = target_image(size, seed)
    cam = ss.pinhole(np.eye(4), 2.0 * size, size, size)
    model = TilePredictor(tiles, tiles, p=p, seed=seed).train()
    raster = gs.Rasterizer(cam, 0, tiles * tiles * model.per_tile)
    ws = _workspace(gs.gs_loss_workspace_bytes(size, size))
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for step in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = RenderLoss.apply(*model(target, cam), raster, target, ws)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if log and (step % 20 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {loss.item():.4f}")
    gs.gs_attention_status()
    return [float(x) for x in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--size", type=int, default=128, help="side of the image, a multiple of 16")
    args = ap.parse_args()
    train(args.steps, args.size // TILE * TILE, log=print)


if __name__ == "__main__":
    main()
