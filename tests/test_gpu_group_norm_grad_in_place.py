"""Group norm's gradient written over the output's gradient (grad_x may be grad_out
itself in the C ABI), and its output over x: bit for bit what separate buffers
give, in every form of the kernels; a piece that repeats channels of its
neighbour's workgroup must not take or leave what the other one has written."""
import ctypes

import pytest
import torch

from deformable_convolution_amd import dc1d, sequence
from deformable_convolution_amd.dc1d import _desc, _ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16

SHAPES = [
    # held: a group's lanes in one wave, whole pieces, one odd group a slab, several odd groups
    ((50, 512), 4), ((2, 784, 64), 4), ((70, 890), 1), ((3, 200, 99), 3), ((3, 257, 255), 17),
    # last slabs of fewer channels than a piece (bf16; fp32), and of a few more
    ((40, 300, 333), 111), ((40, 300, 345), 115), ((2, 300, 165), 33),
    # several samples a workgroup
    ((400, 2, 21), 7), ((3000, 333), 111),
    # in parts: channels in one tile and in several, off a piece's size; a sample to several workgroups
    ((2, 6000, 99), 33), ((2, 5000, 64), 1), ((1, 600, 4105), 5), ((1, 70, 2053), 1), ((2, 40, 8203), 13), ((520, 601, 36), 1), ((520, 601, 37), 1),
]


def backward_over(x, groups, go, mean, rstd, w, b, lens, need_params=True):
    """dc1d_group_norm_backward with grad_x = grad_out = go."""
    lib, n, C = dc1d.load_library(), ctypes.c_size_t(0), x.shape[-1]
    gw, gb = (torch.empty(C, dtype=x.dtype, device=DEV) if need_params else None for _ in range(2))
    dx, dw, db, dl, dg, dm, dr, dgw, dgb = map(_desc, (x, w, b, lens, go, mean, rstd, gw, gb))
    if dl is not None:
        dl.dtype = 2  # DC1D_I32
    i64 = ctypes.c_int64
    assert lib.dc1d_group_norm_backward_workspace_bytes(_ref(dx), i64(groups), int(need_params), ctypes.byref(n)) == 0
    ws = torch.empty(max(n.value, 1), dtype=torch.uint8, device=DEV)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    status = lib.dc1d_group_norm_backward(_ref(dx), _ref(dw), _ref(db), _ref(dl), _ref(dg), _ref(dm), _ref(dr), _ref(dg), _ref(dgw), _ref(dgb),
                                          i64(groups), 2, ctypes.c_void_p(ws.data_ptr() if n.value else None), ctypes.c_size_t(n.value), stream)
    assert status == 0
    return {"x": go, "weight": gw, "bias": gb}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_over_the_output_s_gradient(shape, groups, dtype):
    print("group norm in place", shape, groups, dtype, flush=True)
    gen, C = torch.Generator(device=DEV).manual_seed(1), shape[-1]
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    x, go, w, b = rand(*shape), rand(*shape), rand(C), rand(C)
    some = None
    if len(shape) == 3:
        some = torch.full(shape[:1], shape[1] - 1, dtype=torch.int32, device=DEV)
        some[-1] = shape[1] // 2
    for lens in (None, some)[:1 if some is None else 2]:
        y, mean, rstd = sequence.group_norm(x, groups, w, b, activation="silu", lens=lens, with_stats=True)
        want = sequence.group_norm_backward(x, groups, go, mean, rstd, w, b, "silu", lens)
        for _ in range(5):
            same = x.clone()
            sequence.group_norm(same, groups, w, b, activation="silu", lens=lens, out=same)
            assert torch.equal(same, y)
            got = backward_over(x, groups, go.clone(), mean, rstd, w, b, lens)
            assert all(torch.equal(got[n], want[n]) for n in want)
        assert torch.equal(backward_over(x, groups, go.clone(), mean, rstd, w, b, lens, False)["x"], want["x"])
