"""What attention's mask leaves out is not used, whatever it holds: keys that
no query sees (ahead of a window, past the last query, past the lengths), and
queries that see no key."""
import pytest
import torch

from deformable_convolution_amd import sequence
from oracle import sequence as ref
from test_gpu_sequence import BF16, DEV, F32, att_inputs, i32, mask_of

pytestmark = pytest.mark.gpu


def cycle(B, *v):
    return tuple(v[i % len(v)] for i in range(B))


def gradients(q, k, v, g, mask):
    out, lse = sequence.attention(q, k, v, with_lse=True, **mask)
    return out, lse, sequence.attention_backward(q, k, v, out, lse, g, **mask)


def junk_of(dtype):
    return float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min


# B, Lq, Lk, Hq, Hkv, D, mask, kernel
KEYS = [
    (3, 1, 300, 4, 2, 64, dict(causal=True, window=33, q_start=(299, 150, 40)), "attention_keys"),
    (2, 1, 4096, 8, 1, 128, dict(causal=True, window=100, q_start=(4000, 777)), "attention_keys"),
    (2, 40, 300, 4, 2, 64, dict(causal=True, window=33, q_start=(250, 101)), "attention_keys"),
    (2, 5, 200, 6, 1, 80, dict(window=20, q_start=(90, 61)), "attention_keys"),
    (2, 9, 200, 3, 1, 20, dict(causal=True, q_start=(90, 61)), "attention_keys"),
    (2, 300, 900, 2, 1, 100, dict(causal=True, window=70, q_start=(333, 500)), "attention_keys"),
    (32, 40, 300, 8, 8, 64, dict(causal=True, window=33, q_start=cycle(32, 250, 101, 37)), "attention_rows"),
    (32, 40, 300, 8, 8, 128, dict(window=50, q_start=cycle(32, 200, 101, 131)), "attention_rows"),
    (32, 40, 300, 8, 8, 20, dict(causal=True, window=33, kv_lens=cycle(32, 290, 140), q_start=cycle(32, 250, 101)), "attention_rows"),
]


@pytest.mark.parametrize("spread", [False, True], ids=["near", "far"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", KEYS, ids=lambda c: "-".join(str(v) for v in c[:6]) + "-" + "-".join(c[6]))
def test_keys_that_no_query_sees(case, dtype, spread):
    """spread: rows off every alignment, which are staged another way."""
    print("unseen keys", case, dtype, spread, flush=True)
    B, Lq, Lk, Hq, Hkv, D = case[:6]
    mask = mask_of(case[6])
    q, k, v, g = att_inputs(61, *case[:6], dtype)
    unseen = ~ref.visible(B, Lq, Lk, device=DEV, **mask).any(1)
    assert unseen.any()

    def place(t):
        if not spread:
            return t
        wide = torch.zeros(t.shape[:3] + (D + 3,), dtype=dtype, device=DEV)
        wide[..., 1:D + 1] = t
        return wide[..., 1:D + 1]

    assert sequence.attention_plan(q, k, v)["kernel"] == case[7]
    out, lse, grads = gradients(q, place(k), place(v), g, mask)
    assert not torch.isnan(out).any()
    for junk in junk_of(dtype):
        kj, vj = k.clone(), v.clone()
        kj[unseen], vj[unseen] = junk, junk
        o2, l2, g2 = gradients(q, place(kj), place(vj), g, mask)
        assert torch.equal(o2, out) and torch.equal(l2, lse), junk
        assert all(torch.equal(g2[n], grads[n]) for n in "qkv"), junk
    assert not grads["k"][unseen].any() and not grads["v"][unseen].any()


# B, Lq, Lk, Hq, Hkv, D, mask
QUERIES = [
    (2, 65, 63, 4, 2, 64, dict(causal=True)),
    (2, 90, 40, 6, 2, 128, dict(causal=True)),
    (1, 300, 170, 5, 1, 64, dict(causal=True)),
    (3, 50, 70, 2, 1, 20, dict(kv_lens=(70, 0, 13), causal=True, q_start=(-20, 20, -37))),
    (2, 45, 60, 4, 1, 80, dict(window=9, q_start=(-30, 45))),
    (2, 45, 60, 4, 1, 33, dict(window=9, causal=True, q_start=(-30, 45))),
    (32, 65, 40, 8, 8, 64, dict(causal=True)),
    (4, 520, 500, 2, 2, 32, dict(causal=True)),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", QUERIES, ids=lambda c: "-".join(str(v) for v in c[:6]) + "-" + "-".join(c[6]))
def test_queries_that_see_nothing(case, dtype):
    """Padding: their results are 0, and what q and grad_out hold there reaches no gradient."""
    print("queries that see nothing", case, dtype, flush=True)
    mask = mask_of(case[6])
    q, k, v, g = att_inputs(62, *case[:6], dtype)
    blind = ~ref.visible(case[0], case[1], case[2], device=DEV, **mask).any(2)
    assert blind.any() and not blind.all()
    out, lse, grads = gradients(q, k, v, g, mask)
    for junk in junk_of(dtype):
        qj, gj = q.clone(), g.clone()
        qj[blind], gj[blind] = junk, junk
        o2, l2, g2 = gradients(qj, k, v, gj, mask)
        assert torch.equal(o2, out) and torch.equal(l2, lse), junk
        assert all(torch.equal(g2[n], grads[n]) for n in "qkv"), junk
    assert not out[blind].any() and not grads["q"][blind].any()
