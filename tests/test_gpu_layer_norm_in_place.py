"""Layer norm's gradients written over the output's gradient, which the C ABI
allows: the same bits as apart from it, and nothing around them touched."""
import ctypes
import math

import pytest
import torch

from deformable_convolution_amd import dc1d, sequence
from test_gpu_sequence import BF16, DEV, F32, LN_SHAPES, ODD_SHAPES, ln_inputs

pytestmark = pytest.mark.gpu

REREAD = [(2, 20001), (3, 40000), (1, 2100, 100), (2, 4100, 33), (1, 2049, 65), (3, 1500, 3), (2, 1100, 5)]  # a pass a sum


def backward_over(x, go, mean, rstd, w):
    """dc1d_layer_norm_backward with grad_x = grad_out: grad_weight and grad_bias."""
    lib = dc1d.load_library()
    gw, gb = torch.empty_like(w), torch.empty_like(w)
    d = {n: dc1d._desc(t) for n, t in (("x", x), ("w", w), ("g", go), ("mean", mean), ("rstd", rstd), ("gw", gw), ("gb", gb))}
    ref = lambda n: ctypes.byref(d[n])  # noqa: E731
    need = ctypes.c_size_t()
    assert lib.dc1d_layer_norm_backward_workspace_bytes(ref("x"), 1, ctypes.byref(need)) == dc1d.OK
    ws = torch.empty(max(need.value, 1), dtype=torch.uint8, device=DEV)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    status = lib.dc1d_layer_norm_backward(ref("x"), ref("w"), ref("g"), ref("mean"), ref("rstd"), ref("g"), ref("gw"), ref("gb"),
                                          ctypes.c_void_p(ws.data_ptr()), need, stream)
    assert status == dc1d.OK
    return gw, gb


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", list(dict.fromkeys(LN_SHAPES + ODD_SHAPES + REREAD)))
def test_grad_x_over_grad_out(shape, dtype):
    print("layer norm gradients in place", shape, dtype, flush=True)
    n = math.prod(shape)
    x, w, _, go = ln_inputs(shape, dtype, 13, 0.5)
    for start in (0, 17):  # aligned, and off every alignment, NaN around them
        def amid(t):
            store = torch.full((n + 64,), float("nan"), dtype=dtype, device=DEV)
            store[start:start + n] = t.reshape(-1)
            return store[start:start + n].view(shape), store

        (ox, _), (og, sg) = amid(x), amid(go)
        _, mean, rstd = sequence.layer_norm(ox, w, with_stats=True)
        want = sequence.layer_norm_backward(ox, og, mean, rstd, w)
        gw, gb = backward_over(ox, og, mean, rstd, w)
        assert torch.equal(og, want["x"]) and torch.equal(gw, want["weight"]) and torch.equal(gb, want["bias"])
        assert torch.isnan(sg[:start]).all() and torch.isnan(sg[start + n:]).all()
