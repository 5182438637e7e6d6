"""Attention's gradients where their workgroups are more than one launch holds."""
import pytest
import torch

from deformable_convolution_amd import sequence

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("Lk,D", [(1, 8), (129, 1)])  # with the queries' 2^24 + 2 and 3 (2^23 + 1) workgroups
def test_attention_gradients_of_many_batches(Lk, D):
    B = (1 << 23) + 1
    print("attention gradients", B, Lk, D, flush=True)
    gen = torch.Generator(device=DEV).manual_seed(1)
    dtype = torch.bfloat16
    rand = lambda n: torch.randn((B, n, 1, D), generator=gen, dtype=dtype, device=DEV)  # noqa: E731
    q, k, v, g = rand(1), rand(Lk), rand(Lk), rand(1)
    out, lse = sequence.attention(q, k, v, with_lse=True)
    grads = {n: torch.full_like(t, float("nan")) for n, t in (("q", q), ("k", k), ("v", v))}
    sequence.attention_backward(q, k, v, out, lse, g, grads=grads)
    for n in "qkv":
        assert not torch.isnan(grads[n]).any(), n  # every element was written
    half = (1 << 22) + 1
    at = torch.tensor([0, 1, 2, 1000003, half - 2, half - 1, half, half + 1, B - 4099, B - 9, B - 2, B - 1], device=DEV)
    # the same bits as the same batches by themselves, in a call of one launch
    some = sequence.attention_backward(*(t[at].contiguous() for t in (q, k, v, out, lse, g)))
    for n in "qkv":
        assert torch.equal(grads[n][at], some[n]), n
