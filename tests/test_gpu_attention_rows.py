"""The attention kernel of full batches (128 rows a workgroup), which serves
calls with at least one such workgroup a compute unit, against the float64
forms: the masks, sizes, layouts and junk that test_gpu_sequence.py gives to
smaller calls, which another kernel serves.  Every call here is checked to be
of this kernel.  Tolerances are those of test_gpu_sequence.py."""
import math

import pytest
import torch

from deformable_convolution_amd import sequence
from oracle import sequence as ref
from test_gpu_sequence import BF16, DEV, F32, U32, att_bound, att_inputs, i32, mask_of, ref_mask, within

pytestmark = pytest.mark.gpu


def attention(q, k, v, **kw):
    plan = sequence.attention_plan(q, k, v)
    assert plan["kernel"] == "attention_rows" and plan["splits"] == 1, plan
    return sequence.attention(q, k, v, **kw)


def cycle(B, *v):
    """One value a batch, in turn."""
    return tuple(v[i % len(v)] for i in range(B))


WILD = (2 ** 31 - 1, -2 ** 31, 2 ** 30, -2 ** 30)

# B, Lq, Lk, Hq, Hkv, D, mask
ROWS = [
    (32, 33, 63, 8, 8, 64, {}),
    (32, 33, 1, 8, 8, 64, dict(causal=True)),
    (32, 40, 0, 8, 8, 64, {}),                               # no keys at all
    (32, 128, 128, 8, 8, 128, dict(causal=True)),
    (16, 129, 257, 8, 8, 64, dict(causal=True)),
    (32, 83, 83, 8, 8, 64, {}),
    (32, 65, 63, 8, 8, 32, dict(causal=True)),               # the first queries see nothing
    (32, 64, 64, 8, 8, 20, dict(causal=True)),
    (64, 70, 100, 4, 4, 80, dict(window=17)),
    (64, 40, 90, 4, 4, 100, dict(causal=True, window=9)),
    (64, 50, 50, 4, 4, 96, dict(window=1)),
    (64, 45, 70, 4, 4, 33, dict(causal=True)),
    (256, 34, 5, 1, 1, 7, {}),
    (256, 35, 40, 1, 1, 1, dict(causal=True)),
    (43, 43, 70, 9, 3, 64, dict(causal=True)),               # three heads share a key head; 129 rows
    (52, 43, 70, 15, 5, 128, dict(causal=True, window=20)),
    (256, 3, 90, 16, 1, 64, dict(causal=True)),
    (128, 7, 33, 14, 2, 64, dict(causal=True)),
    (16, 100, 700, 16, 16, 64, dict(causal=True)),
    (2, 1024, 1030, 16, 16, 64, dict(causal=True, window=300)),
    (1, 2048, 700, 16, 16, 32, dict(causal=True)),           # most rows see nothing
    (32, 50, 70, 8, 8, 64, dict(kv_lens=cycle(32, 70, 0, 13, 64, 65, 1, 63, 99, -3))),
    (32, 50, 70, 8, 8, 128, dict(kv_lens=cycle(32, 64, 1, 65, 0), causal=True)),
    (32, 40, 300, 8, 8, 64, dict(kv_lens=cycle(32, 300, 40, 4, 255, 257), causal=True, q_start=cycle(32, 260, 0, -5, 215, 217))),
    (32, 40, 200, 8, 8, 64, dict(kv_lens=cycle(32, 200, 90, 130), causal=True, window=33, q_start=cycle(32, 160, 50, 90))),
    (32, 40, 90, 8, 8, 64, dict(q_start=cycle(32, -40, 1000, 60, *WILD), window=30)),
    (32, 40, 90, 8, 8, 64, dict(q_start=cycle(32, -40, 1000, 60, *WILD), causal=True)),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(str(v) for v in c[:6]) + "-" + "-".join(c[6]))
def test_attention(case, dtype):
    print("attention rows", case, dtype, flush=True)
    shape, mask = case[:6], mask_of(case[6])
    q, k, v, _ = att_inputs(51, *shape, dtype)
    out, lse = attention(q, k, v, with_lse=True, **mask)
    wo, wl, spread = ref.attention(q, k, v, **ref_mask(mask, shape[2]))
    within(lse, wl, 64 * U32 * (4 + wl.abs().nan_to_num(0, 0, 0)), "lse")
    within(out, wo, att_bound(wo, spread, dtype), "out")
    assert torch.equal(out, attention(q, k, v, **mask))
    assert not out[(wl == -math.inf).transpose(1, 2)].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 20])
def test_layouts(D, dtype):
    """Slices of one buffer, heads ahead of positions, a repeated key head: the same bits as contiguous inputs; and
    storage off every alignment."""
    B, Lq, Lk, Hq, Hkv = 32, 70, 90, 16, 8
    q, k, v, _ = att_inputs(52, B, Lq, Lk, Hq, Hkv, D, dtype)
    out, lse = attention(q, k, v, causal=True, with_lse=True)
    kv = torch.full((B, Lk, 2 * Hkv + 1, D), float("nan"), dtype=dtype, device=DEV)
    kv[:, :, :Hkv], kv[:, :, Hkv:2 * Hkv] = k, v
    assert torch.equal(attention(q, kv[:, :, :Hkv], kv[:, :, Hkv:2 * Hkv], causal=True), out)
    t = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    o = t(torch.empty_like(q))
    assert attention(t(q), t(k), t(v), causal=True, out=o) is o and torch.equal(o, out)
    both = torch.full((B, Lq, 2 * Hq, D), 3.0, dtype=dtype, device=DEV)  # the output beside its queries
    both[:, :, :Hq] = q
    attention(both[:, :, :Hq], k, v, causal=True, out=both[:, :, Hq:])
    assert torch.equal(both[:, :, Hq:], out) and torch.equal(both[:, :, :Hq], q)
    one = attention(q, k[:, :, :1].expand_as(k), v[:, :, :1].expand_as(v), causal=True)
    assert torch.equal(one, attention(q, k[:, :, :1].repeat(1, 1, Hkv, 1), v[:, :, :1].repeat(1, 1, Hkv, 1), causal=True))

    def off(x):
        wide = torch.full(x.shape[:3] + (D + 3,), float("nan"), dtype=dtype, device=DEV)
        wide[..., 1:D + 1] = x
        return wide

    wq, wk, wv, wo = off(q), off(k), off(v), off(torch.zeros_like(q))
    got, l2 = attention(wq[..., 1:D + 1], wk[..., 1:D + 1], wv[..., 1:D + 1], causal=True, out=wo[..., 1:D + 1], with_lse=True)
    want, wl, spread = ref.attention(q, k, v, causal=True)
    within(got, want, att_bound(want, spread, dtype), "unaligned")
    within(l2, wl, 64 * U32 * (4 + wl.abs()), "unaligned lse")
    assert torch.isnan(wo[..., 0]).all() and torch.isnan(wo[..., D + 1:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_what_lies_past_the_lengths_is_ignored(dtype):
    B, Lq, Lk, H, D = 32, 70, 150, 8, 64
    q, k, v, _ = att_inputs(53, B, Lq, Lk, H, H, D, dtype)
    lens = i32(*cycle(B, 150, 101, 64, 1, 0, 129))
    kw = dict(kv_lens=lens, q_start=lens - Lq, causal=True)
    out, lse = attention(q, k, v, with_lse=True, **kw)
    past = torch.arange(Lk, device=DEV).view(1, Lk) >= lens.view(B, 1)
    for junk in (float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min):
        kj, vj = k.clone(), v.clone()
        kj[past], vj[past] = junk, junk
        o2, l2 = attention(q, kj, vj, with_lse=True, **kw)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_nan_reaches_its_row_only():
    q, k, v, _ = att_inputs(54, 32, 70, 70, 8, 8, 64, BF16)
    clean = attention(q, k, v)
    q[5, 33, 1, 5] = float("nan")
    out = attention(q, k, v)
    assert out[5, 33, 1].isnan().all()
    out[5, 33, 1] = clean[5, 33, 1]
    assert torch.equal(out, clean)


def test_extreme_scores():
    q, k, v, _ = att_inputs(55, 32, 96, 96, 8, 8, 64, F32)
    for qs, ks in ((q * 30, k * 30), (q.abs() * 10, -k.abs() * 10)):
        out, lse = attention(qs, ks, v, with_lse=True)
        wo, wl, spread = ref.attention(qs, ks, v)
        terms = torch.matmul(qs.double().abs().transpose(1, 2).contiguous(), ks.double().abs().permute(0, 2, 3, 1).contiguous())
        big = float(terms.max()) / math.sqrt(64)
        within(lse, wl, 4 * U32 * big, "lse")
        within(out, wo, 16 * U32 * big * spread + 1e-6, "out")


def test_offsets_past_32_bits():
    """Keys so far apart that the last ones lie past 2^31 elements, shared by every batch and head."""
    B, Lq, Lk, H, D = 32, 70, 65, 8, 64
    row = (1 << 31) // 50 // 8 * 8
    store = torch.zeros(row * Lk + D, dtype=BF16, device=DEV)
    q, k, v, _ = att_inputs(56, B, Lq, Lk, H, H, D, BF16)
    k, v = k[:1, :, :1].expand_as(k), v[:1, :, :1].expand_as(v)
    far = store.as_strided((B, Lk, H, D), (0, row, 0, 1))
    far[0, :, 0].copy_(k[0, :, 0])
    want = attention(q, k, v, causal=True)
    assert torch.equal(attention(q, far, v, causal=True), want)
    assert torch.equal(attention(q, k, far, causal=True), attention(q, k, k, causal=True))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeats_streams_and_graphs(dtype):
    q, k, v, _ = att_inputs(57, 32, 150, 300, 8, 8, 64, dtype)
    call = lambda: attention(q, k, v, causal=True, with_lse=True)  # noqa: E731
    want = [t.clone() for t in call()]
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(want, call()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        call()


def test_the_smaller_calls_are_of_the_other_kernel():
    """One workgroup below one a compute unit, and single positions."""
    cus = torch.cuda.get_device_properties(DEV).multi_processor_count
    for B, Lq, kernel in ((cus, 33, "attention_rows"), (cus - 1, 33, "attention_keys"), (cus, 32, "attention_keys"),
                          (4 * cus, 1, "attention_keys")):
        q, k, v, _ = att_inputs(58, B, Lq, 40, 1, 1, 64, BF16)
        plan = sequence.attention_plan(q, k, v)
        assert plan["kernel"] == kernel, (B, Lq, plan)
        wo, _, spread = ref.attention(q, k, v)
        within(sequence.attention(q, k, v), wo, att_bound(wo, spread, BF16), "out")
