"""hr_reduce_rmsnorm and hr_rmsnorm_grad refuse bad arguments before any device
call (CPU): the addresses below are never dereferenced."""
import ctypes

import pytest

from message_fp16_all_amd import hr

BASE = 0x7F0000000000
STEP = 1 << 24


def at(i):
    return BASE + i * STEP


def norm_args(**over):
    a = hr.hr_rmsnorm_args()
    a.inputs[0], a.inputs[1] = at(0), at(1)
    a.G, a.rows, a.hidden, a.eps = 2, 16, 128, 1e-6
    a.residual, a.weight, a.residual_out, a.out = at(2), at(3), at(4), at(5)
    a.codes, a.scales, a.rstd = at(6), at(7), at(8)
    for k, v in over.items():
        if k == "input1":
            a.inputs[1] = v
        else:
            setattr(a, k, v)
    return a


def both(args, f16, bf16):
    got = {f16(args, 0), bf16(args, 0)}
    assert len(got) == 1
    return got.pop()


def norm(**over):
    return both(norm_args(**over), hr.hr_reduce_rmsnorm_f16, hr.hr_reduce_rmsnorm_bf16)


def test_structs_match_their_packed_form():
    assert ctypes.sizeof(hr.hr_rmsnorm_args) == hr._NORM.size
    assert ctypes.sizeof(hr.hr_rmsnorm_grad_args) == hr._NORM_GRAD.size


@pytest.mark.parametrize("over,status", [
    (dict(G=0), hr.HR_ERR_INVALID_ARG), (dict(G=17), hr.HR_ERR_INVALID_ARG),
    (dict(hidden=0), hr.HR_ERR_INVALID_ARG), (dict(eps=-1.0), hr.HR_ERR_INVALID_ARG),
    (dict(eps=float("nan")), hr.HR_ERR_INVALID_ARG),
    (dict(group=16), hr.HR_ERR_INVALID_ARG), (dict(group=-32), hr.HR_ERR_INVALID_ARG),
    (dict(group=256), hr.HR_ERR_INVALID_ARG),
    (dict(input1=None), hr.HR_ERR_INVALID_ARG), (dict(codes=None), hr.HR_ERR_INVALID_ARG),
    (dict(scales=None), hr.HR_ERR_INVALID_ARG),
    (dict(out=None, residual_out=None, codes=None, scales=None, rstd=None), hr.HR_ERR_INVALID_ARG),
    (dict(hidden=hr.HR_RMSNORM_MAX_HIDDEN + 1), hr.HR_ERR_TOO_LARGE), (dict(rows=1 << 31), hr.HR_ERR_TOO_LARGE),
    (dict(input_stride=127), hr.HR_ERR_INVALID_ARG), (dict(out_stride=100), hr.HR_ERR_INVALID_ARG),
    (dict(residual_stride=1), hr.HR_ERR_INVALID_ARG), (dict(residual_out_stride=1), hr.HR_ERR_INVALID_ARG),
    (dict(codes_stride=1), hr.HR_ERR_INVALID_ARG), (dict(group=32, scales_stride=3), hr.HR_ERR_INVALID_ARG),
    (dict(input_stride=1 << 62), hr.HR_ERR_INVALID_ARG),
    (dict(input1=at(1) + 1), hr.HR_ERR_ALIGNMENT), (dict(residual=at(2) + 1), hr.HR_ERR_ALIGNMENT),
    (dict(out=at(5) + 1), hr.HR_ERR_ALIGNMENT), (dict(residual_out=at(4) + 1), hr.HR_ERR_ALIGNMENT),
    (dict(scales=at(7) + 2), hr.HR_ERR_ALIGNMENT), (dict(rstd=at(8) + 2), hr.HR_ERR_ALIGNMENT),
    (dict(weight=at(3) + 1), hr.HR_ERR_ALIGNMENT), (dict(weight=at(3) + 2, weight_f32=1), hr.HR_ERR_ALIGNMENT),
    # overlaps: an output half over an input, over another output, over the weight
    (dict(out=at(0) + 64), hr.HR_ERR_INVALID_ARG), (dict(residual_out=at(1) + 256), hr.HR_ERR_INVALID_ARG),
    (dict(out=at(4)), hr.HR_ERR_INVALID_ARG), (dict(codes=at(5) + 17), hr.HR_ERR_INVALID_ARG),
    (dict(codes=at(0)), hr.HR_ERR_INVALID_ARG), (dict(scales=at(2) + 4), hr.HR_ERR_INVALID_ARG),
    (dict(out=at(3)), hr.HR_ERR_INVALID_ARG), (dict(rstd=at(7)), hr.HR_ERR_INVALID_ARG),
    # the same address with another stride is not in place
    (dict(out=at(0), out_stride=256), hr.HR_ERR_INVALID_ARG),
    # one row: the weight is no input to take the place of
    (dict(rows=1, out=at(3)), hr.HR_ERR_INVALID_ARG), (dict(rows=1, residual_out=at(3)), hr.HR_ERR_INVALID_ARG),
    # interleaved columns that meet
    (dict(input_stride=256, out=at(0) + 254, out_stride=256), hr.HR_ERR_INVALID_ARG),
])
def test_norm_refusals(over, status):
    assert norm(**over) == status


def test_norm_refuses_no_struct_and_takes_no_rows():
    lib = hr.load()
    assert lib.hr_reduce_rmsnorm_f16(None, None) == hr.HR_ERR_INVALID_ARG
    assert lib.hr_rmsnorm_grad_bf16(None, None) == hr.HR_ERR_INVALID_ARG
    assert norm(rows=0) == hr.HR_OK


def grad_args(**over):
    a = hr.hr_rmsnorm_grad_args()
    a.dy, a.h, a.rstd, a.weight, a.dresidual, a.dx, a.dweight = (at(i) for i in range(7))
    a.rows, a.hidden = 5000, 64
    a.workspace, a.workspace_bytes = at(7), hr.hr_rmsnorm_grad_workspace(5000, 64)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(hidden=0), hr.HR_ERR_INVALID_ARG), (dict(dy=None), hr.HR_ERR_INVALID_ARG),
    (dict(h=None), hr.HR_ERR_INVALID_ARG), (dict(rstd=None), hr.HR_ERR_INVALID_ARG),
    (dict(dx=None), hr.HR_ERR_INVALID_ARG), (dict(workspace=None), hr.HR_ERR_INVALID_ARG),
    (dict(workspace_bytes=hr.hr_rmsnorm_grad_workspace(5000, 64) - 1), hr.HR_ERR_INVALID_ARG),
    (dict(hidden=hr.HR_RMSNORM_MAX_HIDDEN + 1), hr.HR_ERR_TOO_LARGE), (dict(rows=1 << 31), hr.HR_ERR_TOO_LARGE),
    (dict(dy_stride=63), hr.HR_ERR_INVALID_ARG), (dict(h_stride=63), hr.HR_ERR_INVALID_ARG),
    (dict(dx_stride=63), hr.HR_ERR_INVALID_ARG), (dict(dresidual_stride=63), hr.HR_ERR_INVALID_ARG),
    (dict(dx=at(5) + 1), hr.HR_ERR_ALIGNMENT), (dict(dweight=at(6) + 2), hr.HR_ERR_ALIGNMENT),
    (dict(workspace=at(7) + 2), hr.HR_ERR_ALIGNMENT), (dict(rstd=at(2) + 1), hr.HR_ERR_ALIGNMENT),
    (dict(dx=at(0) + 2), hr.HR_ERR_INVALID_ARG), (dict(dx=at(6)), hr.HR_ERR_INVALID_ARG),
    (dict(dweight=at(3)), hr.HR_ERR_INVALID_ARG), (dict(workspace=at(5)), hr.HR_ERR_INVALID_ARG),
    (dict(workspace=at(1) + 8), hr.HR_ERR_INVALID_ARG),
    # one row: neither the weight nor rstd is an input to take the place of
    (dict(rows=1, dx=at(3)), hr.HR_ERR_INVALID_ARG), (dict(rows=1, hidden=2, dx=at(2)), hr.HR_ERR_INVALID_ARG),
])
def test_grad_refusals(over, status):
    assert both(grad_args(**over), hr.hr_rmsnorm_grad_f16, hr.hr_rmsnorm_grad_bf16) == status


def test_grad_workspace_sizes():
    f = hr.hr_rmsnorm_grad_workspace
    assert f(0, 128) == 0 and f(1, 4096) == 0 and f(10, 0) == 0 and f(10, hr.HR_RMSNORM_MAX_HIDDEN + 1) == 0
    assert f(16, 128) == 0                      # one workgroup's rows
    assert f(2, 4096) == 2 * 4096 * 4
    assert f(1 << 20, 8192) == f(1 << 24, 8192)  # bounded by the device, not by the rows
