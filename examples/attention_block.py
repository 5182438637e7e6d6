"""A pre-norm attention block ahead of a deformable convolution: training steps
and decoding position by position, on the package's operators.

    python examples/attention_block.py

The block mixes the whole sequence, the convolution after it samples locally:

    h = layer_norm(x);  q, k, v = heads of h Wqkv;  q, k turned by rotary
    positions;  y = x + attention(q, k, v) Wo;  z = deformable conv1d(y)

x is channels first [B, C, L], as the convolution takes it.  The products
with Wqkv and Wo are torch's; everything else is the package's, gradients
included, none of it through autograd.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from deformable_convolution_amd import dc1d, sequence  # noqa: E402


class Block:
    """The block's sizes, weights and rotary tables."""

    def __init__(self, C, heads, kv_heads, max_len, dtype=torch.float32, device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.C, self.Hq, self.Hkv, self.D = C, heads, kv_heads, C // heads
        rand = lambda *s: (torch.randn(s, generator=gen) / s[-1] ** 0.5).to(device, dtype)  # noqa: E731
        self.norm_w = torch.ones(C, dtype=dtype, device=device)
        self.norm_b = torch.zeros(C, dtype=dtype, device=device)
        self.wqkv = rand((heads + 2 * kv_heads) * self.D, C)
        self.wo = rand(C, C)
        R = self.D // 2
        angle = torch.arange(max_len, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(R, dtype=torch.float64) / R)
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        self.sections = (R,)

    def split(self, qkv):
        """Head slices of one buffer [B, L, Hq + 2 Hkv, D]: no copies."""
        a, b = self.Hq, self.Hq + self.Hkv
        return qkv[:, :, :a], qkv[:, :, a:b], qkv[:, :, b:]

    def turn(self, q, k, positions, inverse=False):
        sequence.rotary(q, k, self.cos, self.sin, positions, self.sections, inverse=inverse, out=(q, k))


def positions(L, device, first=0):
    return torch.arange(first, first + L, dtype=torch.int32, device=device).view(1, L, 1)


def forward(blk, x):
    """y [B, C, L] and what the backward needs of it."""
    B, C, L = x.shape
    h, mean, rstd = sequence.layer_norm(x, blk.norm_w, blk.norm_b, with_stats=True)
    rows = h.transpose(1, 2).reshape(B * L, C)
    qkv = torch.mm(rows, blk.wqkv.t()).view(B, L, -1, blk.D)
    q, k, v = blk.split(qkv)
    blk.turn(q, k, positions(L, x.device))
    out, lse = sequence.attention(q, k, v, causal=True, with_lse=True)
    y = x + torch.mm(out.view(B * L, C), blk.wo.t()).view(B, L, C).transpose(1, 2)
    return y, (x, mean, rstd, rows, qkv, out, lse)


def backward(blk, saved, gy):
    """Gradients of sum(gy * y): a dict of x, norm_w, norm_b, wqkv, wo."""
    x, mean, rstd, rows, qkv, out, lse = saved
    B, C, L = x.shape
    gy_rows = gy.transpose(1, 2).reshape(B * L, C)
    gout = torch.mm(gy_rows, blk.wo).view(B, L, blk.Hq, blk.D)
    gqkv = torch.empty_like(qkv)
    gq, gk, gv = blk.split(gqkv)
    q, k, v = blk.split(qkv)
    sequence.attention_backward(q, k, v, out, lse, gout, causal=True, grads={"q": gq, "k": gk, "v": gv})
    blk.turn(gq, gk, positions(L, x.device), inverse=True)
    flat = gqkv.view(B * L, -1)
    gh = torch.mm(flat, blk.wqkv).view(B, L, C).transpose(1, 2).contiguous()
    norm = sequence.layer_norm_backward(x, gh, mean, rstd, blk.norm_w)
    return {"x": norm["x"] + gy, "norm_w": norm["weight"], "norm_b": norm["bias"],
            "wqkv": torch.mm(flat.t(), rows), "wo": torch.mm(gy_rows.t(), out.view(B * L, C))}


class Cache:
    """Keys and values of up to max_len positions for each of B sequences, and how many each holds."""

    def __init__(self, blk, B, max_len, dtype, device="cuda"):
        self.k = torch.empty((B, max_len, blk.Hkv, blk.D), dtype=dtype, device=device)
        self.v = torch.empty_like(self.k)
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)


def decode(blk, cache, x):
    """One new position x [B, C] of every sequence: y [B, C], the cache one longer."""
    B, C = x.shape
    h = sequence.layer_norm(x, blk.norm_w, blk.norm_b)
    q, k, v = blk.split(torch.mm(h, blk.wqkv.t()).view(B, 1, -1, blk.D))
    blk.turn(q, k, cache.lens.view(B, 1, 1))
    seq, at = torch.arange(B, device=x.device), cache.lens.long()
    cache.k[seq, at], cache.v[seq, at] = k[:, 0], v[:, 0]
    cache.lens += 1
    out = sequence.attention(q, cache.k, cache.v, causal=True, kv_lens=cache.lens, q_start=cache.lens - 1)
    return x + torch.mm(out.view(B, C), blk.wo.t())


def main():
    B, C, L, K, dilation = 16, 512, 128, 16, 3  # the layer's own sizes
    L_out = dc1d.output_length(L, K, dilation=dilation)
    gen = torch.Generator(device="cuda").manual_seed(1)
    blk = Block(C, 8, 2, L)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, target = randn(B, C, L), randn(B, C, L_out)
    offsets, weight, bias = randn(B, 1, L_out, K), randn(C, C, K) / (C * K) ** 0.5, torch.zeros(C, device="cuda")
    rate = 2.0
    for step in range(10):
        y, saved = forward(blk, x)
        y = y.contiguous()
        z = dc1d.forward(y, offsets, weight, bias, dilation=dilation)
        diff = z - target
        print("step %d loss %.5f" % (step, float(diff.square().mean())), flush=True)
        conv = dc1d.backward(y, offsets, weight, 2.0 / diff.numel() * diff, dilation=dilation)
        grads = backward(blk, saved, conv["x"])
        for name in ("norm_w", "norm_b", "wqkv", "wo"):
            getattr(blk, name).sub_(rate * grads[name])
        for t, name in ((offsets, "offsets"), (weight, "weight"), (bias, "bias")):
            t.sub_(rate * conv[name])
    whole, _ = forward(blk, x)
    cache = Cache(blk, B, L, x.dtype)
    steps = torch.stack([decode(blk, cache, x[:, :, i].contiguous()) for i in range(L)], 2)
    print("decoding position by position against the whole sequence: largest difference %.2g"
          % float((steps - whole).abs().max()), flush=True)


if __name__ == "__main__":
    main()
