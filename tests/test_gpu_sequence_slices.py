"""Results written into slices of one buffer, whichever way it is packed: the
same bits as into tensors of their own."""
import pytest
import torch

from deformable_convolution_amd import sequence
from test_gpu_sequence import BF16, DEV, F32, att_inputs, rotary_case

pytestmark = pytest.mark.gpu

B, L, H, D = 2, 37, 3, 64


def packed(how, dtype):
    """Three [B, L, H, D] slices of one buffer, and the buffer."""
    shape = {"heads": (B, L, H, 4, D), "batches": (B, 4, L, H, D), "rows": (B, L, H, 4 * D), "positions": (B, 4 * L, H, D),
             "ahead": (4, B, L, H, D), "transposed": (B, H, L, 4, D)}[how]
    t = torch.full(shape, 3.0, dtype=dtype, device=DEV)
    cut = {"heads": lambda i: t[:, :, :, i], "batches": lambda i: t[:, i], "rows": lambda i: t[..., i * D:(i + 1) * D],
           "positions": lambda i: t[:, i * L:(i + 1) * L], "ahead": lambda i: t[i],
           "transposed": lambda i: t[:, :, :, i].transpose(1, 2)}[how]
    return [cut(i) for i in range(3)], cut(3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("how", ["heads", "batches", "rows", "positions", "ahead", "transposed"])
def test_packed_results(how, dtype):
    q, k, v, g = att_inputs(71, B, L, L, H, H, D, dtype)
    out, lse = sequence.attention(q, k, v, causal=True, with_lse=True)
    want = sequence.attention_backward(q, k, v, out, lse, g, causal=True)
    parts, rest = packed(how, dtype)
    sequence.attention_backward(q, k, v, out, lse, g, causal=True, grads=dict(zip("qkv", parts)))
    assert all(torch.equal(p, want[n]) for p, n in zip(parts, "qkv"))
    assert (rest == 3.0).all()
    # the output beside its inputs, then q and k turned in place
    for p, t in zip(parts, (q, k, v)):
        p.copy_(t)
    assert torch.equal(sequence.attention(*parts, causal=True, out=rest), out)
    _, _, cos, sin, pos = rotary_case(72, B, L, H, H, D, (12, 20), dtype)
    turned = sequence.rotary(q, k, cos, sin, pos, (12, 20))
    sequence.rotary(parts[0], parts[1], cos, sin, pos, (12, 20), out=(parts[0], parts[1]))
    assert torch.equal(parts[0], turned[0]) and torch.equal(parts[1], turned[1]) and torch.equal(parts[2], v)
    assert torch.equal(rest, out)
    with pytest.raises(ValueError):
        sequence.attention(*parts, out=parts[1])
