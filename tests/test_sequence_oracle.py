"""The sequence operators' float64 forms (oracle/sequence.py) pinned on the
CPU: against torch's own layer norm and softmax in float64, closed forms, and
central differences of the forward for every gradient (no GPU needed)."""
import math

import pytest
import torch

from oracle import sequence as ref

F8 = torch.float64


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F8)


def slope(f, at, i, d, h=1e-5):
    up, down = list(at), list(at)
    up[i], down[i] = at[i] + h * d, at[i] - h * d
    return float((f(*up) - f(*down)) / (2 * h))


@pytest.mark.parametrize("shape", [(4, 9), (2, 9, 5), (2, 6, 3, 4)])
def test_layer_norm(shape):
    x, w, b, g = randn(1, *shape), randn(2, shape[1]), randn(3, shape[1]), randn(4, *shape)
    y, mean, rstd = ref.layer_norm(x, w, b)
    last = torch.nn.functional.layer_norm(x.movedim(1, -1), (shape[1],), w, b, 1e-5).movedim(-1, 1)
    assert torch.allclose(y, last, rtol=0, atol=1e-13)
    assert mean.shape == shape[:1] + shape[2:] == rstd.shape
    grads = ref.layer_norm_backward(x, g, w)
    f = lambda *a: (ref.layer_norm(*a)[0] * g).sum()  # noqa: E731
    for i, key in enumerate(("x", "weight", "bias")):
        d = randn(5 + i, *grads[key].shape)
        assert abs(float((grads[key] * d).sum()) - slope(f, [x, w, b], i, d)) < 1e-8 * shape[1] * 10


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(interleaved):
    B, L, H, D, sections = 2, 3, 2, 14, (2, 0, 4)
    R = sum(sections)
    angle = randn(11, 9, R)
    pos = torch.randint(0, 9, (B, L, 3), generator=torch.Generator().manual_seed(12))
    x = randn(13, B, L, H, D)
    kw = dict(interleaved=interleaved)
    y = ref.rotary(x, angle.cos(), angle.sin(), pos, sections, **kw)
    # lengths of pairs stay, the rest is carried over, the inverse turns back
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), atol=1e-12) and torch.equal(y[..., 2 * R:], x[..., 2 * R:])
    assert torch.allclose(ref.rotary(y, angle.cos(), angle.sin(), pos, sections, inverse=True, **kw), x, atol=1e-12)
    # pair 3 (the second of the third axis' section) as a complex number
    a, b = (6, 7) if interleaved else (3, R + 3)
    z = torch.complex(x[1, 2, 1, a], x[1, 2, 1, b]) * torch.exp(1j * angle[pos[1, 2, 2], 3])
    assert abs(complex(z) - complex(y[1, 2, 1, a], y[1, 2, 1, b])) < 1e-12


def test_attention_against_a_loop():
    B, Lq, Lk, Hq, Hkv, D = 2, 5, 7, 4, 2, 3
    q, k, v = randn(21, B, Lq, Hq, D), randn(22, B, Lk, Hkv, D), randn(23, B, Lk, Hkv, D)
    lens, start = torch.tensor([7, 3]), torch.tensor([2, -2])
    out, lse, _ = ref.attention(q, k, v, causal=True, window=3, kv_lens=lens, q_start=start)
    for b in range(B):
        for i in range(Lq):
            p = int(start[b]) + i
            keys = [j for j in range(int(lens[b])) if j <= p and abs(p - j) < 3]
            for h in range(Hq):
                if not keys:
                    assert float(lse[b, h, i]) == -math.inf and not out[b, i, h].any()
                    continue
                s = torch.stack([q[b, i, h] @ k[b, j, h // 2] / math.sqrt(D) for j in keys])
                want = torch.softmax(s, 0) @ torch.stack([v[b, j, h // 2] for j in keys])
                assert torch.allclose(out[b, i, h], want, atol=1e-12)
                assert abs(float(lse[b, h, i] - s.exp().sum().log())) < 1e-12


@pytest.mark.parametrize("mask", [{}, dict(causal=True), dict(window=2), dict(kv_lens=torch.tensor([6, 0]), causal=True)])
def test_attention_backward(mask):
    B, Lq, Lk, Hq, Hkv, D = 2, 4, 6, 4, 2, 5
    at = [randn(31, B, Lq, Hq, D), randn(32, B, Lk, Hkv, D), randn(33, B, Lk, Hkv, D)]
    g = randn(34, B, Lq, Hq, D)
    grads, bound = ref.attention_backward(*at, g, **mask)
    f = lambda *a: (ref.attention(*a, **mask)[0] * g).sum()  # noqa: E731
    for i, key in enumerate("qkv"):
        d = randn(35 + i, *at[i].shape)
        assert abs(float((grads[key] * d).sum()) - slope(f, at, i, d)) < 1e-7
        assert bound[key].shape == grads[key].shape and (bound[key] >= 0).all()


def test_attention_never_looks_past_the_lengths():
    q, k, v, g = randn(41, 1, 3, 2, 4), randn(42, 1, 5, 1, 4), randn(43, 1, 5, 1, 4), randn(44, 1, 3, 2, 4)
    lens = torch.tensor([2])
    want = ref.attention(q, k, v, kv_lens=lens)[0]
    k[:, 2:], v[:, 2:] = math.nan, math.inf
    assert torch.equal(ref.attention(q, k, v, kv_lens=lens)[0], want)
    grads, _ = ref.attention_backward(q, k, v, g, kv_lens=lens)
    assert all(torch.isfinite(t).all() for t in grads.values()) and not grads["k"][:, 2:].any()
