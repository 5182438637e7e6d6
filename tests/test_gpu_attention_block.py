"""The example's attention block (examples/attention_block.py): its hand-written
backward against float64 autograd of the plain block, decoding against the
whole sequence, and a training step through the deformable convolution."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def plain(x, norm_w, norm_b, wqkv, wo, blk):
    """The block in float64 from torch's elementary operations."""
    B, C, L = x.shape
    h = x - x.mean(1, keepdim=True)
    h = h * (h.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * norm_w[:, None] + norm_b[:, None]
    heads = (h.transpose(1, 2) @ wqkv.t()).view(B, L, -1, blk.D).transpose(1, 2)
    R = blk.D // 2
    c, s = blk.cos[:L].double(), blk.sin[:L].double()
    turn = lambda t: torch.cat([t[..., :R] * c - t[..., R:] * s, t[..., :R] * s + t[..., R:] * c], -1)  # noqa: E731
    G = blk.Hq // blk.Hkv
    q = turn(heads[:, :blk.Hq])
    k = turn(heads[:, blk.Hq:blk.Hq + blk.Hkv]).repeat_interleave(G, 1)
    v = heads[:, blk.Hq + blk.Hkv:].repeat_interleave(G, 1)
    S = q @ k.transpose(2, 3) * blk.D ** -0.5
    S = S.masked_fill(torch.ones((L, L), dtype=torch.bool, device=x.device).triu(1), -torch.inf)
    out = (torch.softmax(S, -1) @ v).transpose(1, 2).reshape(B, L, C)
    return x + (out @ wo.t()).transpose(1, 2)


def case(B=3, C=128, L=37):
    blk = example.Block(C, 4, 2, 64)
    x = torch.randn((B, C, L), generator=torch.Generator().manual_seed(5)).cuda()
    blk.norm_w += 0.1 * torch.randn(C, generator=torch.Generator().manual_seed(6)).cuda()
    return blk, x


def test_forward_and_backward():
    blk, x = case()
    y, saved = example.forward(blk, x)
    gy = torch.randn(y.shape, generator=torch.Generator().manual_seed(7)).cuda()
    got = example.backward(blk, saved, gy)
    names = ("x", "norm_w", "norm_b", "wqkv", "wo")
    at = [t.double().requires_grad_() for t in (x, blk.norm_w, blk.norm_b, blk.wqkv, blk.wo)]
    want = plain(*at, blk)
    grads = torch.autograd.grad((want * gy.double()).sum(), at)
    # fp32 sums of up to 128 terms, five operators deep: 1e-4 of the largest value
    assert (y.double() - want).abs().max() <= 1e-4 * want.abs().max()
    for name, g in zip(names, grads):
        assert (got[name].double() - g).abs().max() <= 1e-4 * g.abs().max(), name


def test_decoding_matches_the_whole_sequence():
    blk, x = case()
    whole, _ = example.forward(blk, x)
    cache = example.Cache(blk, x.shape[0], 64, x.dtype)
    cache.k.fill_(float("nan"))  # what a fresh cache holds past its lengths is never used
    cache.v.fill_(float("nan"))
    for i in range(x.shape[2]):
        y = example.decode(blk, cache, x[:, :, i].contiguous())
        assert (y - whole[:, :, i]).abs().max() <= 1e-4 * whole.abs().max(), i


def test_example_runs(capsys):
    example.main()
    out = capsys.readouterr().out
    losses = [float(line.split()[-1]) for line in out.splitlines() if line.startswith("step")]
    assert len(losses) == 10 and losses[-1] < losses[0]
    assert float(out.split()[-1]) < 1e-3
