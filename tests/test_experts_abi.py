"""The experts' entry points refuse bad arguments before any device call (CPU):
the addresses below are never dereferenced."""
import ctypes

import pytest

from message_fp16_all_amd import hr

BASE = 0x7F0000000000
STEP = 1 << 28


def at(i):
    return BASE + i * STEP


def test_structs_match_their_packed_form():
    for c, p in ((hr.hr_experts_gather_args, hr._GATHER), (hr.hr_experts_combine_args, hr._COMBINE),
                 (hr.hr_experts_combine_grad_args, hr._COMBINE_GRAD)):
        assert ctypes.sizeof(c) == p.size


def test_sizes():
    rows, ws = hr.hr_experts_rows, hr.hr_experts_sort_workspace
    assert rows(0, 4, 8, 16) == 0 and rows(5, 0, 8, 1) == 0 and rows(5, 1, 0, 1) == 0 and rows(5, 1, 8, 0) == 0
    assert rows(1 << 62, 32, 8, 1) == 0                         # past the address space
    assert rows(5, 2, 8, 16) == 10 + 8 * 15
    assert ws(1024, 8, 128) == 0 and ws(1025, 8, 128) > 0
    assert ws(1 << 31, 1, 128) == 0 and ws(1 << 20, 8, 1025) == 0
    assert ws(1 << 27, 8, 128) == 256 * 128 * 4                 # bounded by the workgroups


def sort(ids=at(0), tokens=2000, k=8, first=0, experts=64, pad=16, offsets=at(1), order=at(2), rows=None, pos=at(3),
         ws=at(4), ws_bytes=1 << 20):
    if rows is None:
        rows = hr.hr_experts_rows(tokens, k, experts, pad)
    return hr.hr_experts_sort(ids, tokens, k, first, experts, pad, offsets, order, rows, pos, ws, ws_bytes, 0)


@pytest.mark.parametrize("over,status", [
    (dict(k=0), hr.HR_ERR_INVALID_ARG), (dict(first=-1), hr.HR_ERR_INVALID_ARG),
    (dict(experts=0), hr.HR_ERR_INVALID_ARG), (dict(pad=0), hr.HR_ERR_INVALID_ARG),
    (dict(experts=1025), hr.HR_ERR_TOO_LARGE), (dict(k=33), hr.HR_ERR_TOO_LARGE),
    (dict(tokens=1 << 30), hr.HR_ERR_TOO_LARGE), (dict(tokens=1 << 62), hr.HR_ERR_INVALID_ARG),
    (dict(rows=16000 + 64 * 15 - 1), hr.HR_ERR_INVALID_ARG), (dict(rows=1 << 31), hr.HR_ERR_TOO_LARGE),
    (dict(pad=1 << 30), hr.HR_ERR_TOO_LARGE),
    (dict(ids=None), hr.HR_ERR_INVALID_ARG), (dict(offsets=None), hr.HR_ERR_INVALID_ARG),
    (dict(order=None), hr.HR_ERR_INVALID_ARG), (dict(pos=None), hr.HR_ERR_INVALID_ARG),
    (dict(ws=None), hr.HR_ERR_INVALID_ARG), (dict(ws_bytes=16), hr.HR_ERR_INVALID_ARG),
    (dict(ids=at(0) + 2), hr.HR_ERR_ALIGNMENT), (dict(offsets=at(1) + 1), hr.HR_ERR_ALIGNMENT),
    (dict(order=at(2) + 2), hr.HR_ERR_ALIGNMENT), (dict(pos=at(3) + 2), hr.HR_ERR_ALIGNMENT),
    (dict(ws=at(4) + 2), hr.HR_ERR_ALIGNMENT),
    (dict(pos=at(0)), hr.HR_ERR_INVALID_ARG), (dict(order=at(0) + 4), hr.HR_ERR_INVALID_ARG),
    (dict(offsets=at(2) + 8), hr.HR_ERR_INVALID_ARG), (dict(ws=at(3) + 4), hr.HR_ERR_INVALID_ARG)])
def test_sort_refusals(over, status):
    assert sort(**over) == status


def gather(**over):
    a = hr.hr_experts_gather_args()
    a.in_, a.scales, a.out, a.scales_out, a.pos, a.order, a.offsets = (at(i) for i in range(7))
    a.tokens, a.rows, a.row_bytes, a.scales_width, a.k, a.experts = 100, 400, 1024, 8, 4, 16
    for n, v in over.items():
        setattr(a, n, v)
    return hr.hr_experts_gather(a, 0)


@pytest.mark.parametrize("over,status", [
    (dict(row_bytes=0), hr.HR_ERR_INVALID_ARG), (dict(k=0), hr.HR_ERR_INVALID_ARG),
    (dict(k=33), hr.HR_ERR_INVALID_ARG), (dict(in_=None), hr.HR_ERR_INVALID_ARG),
    (dict(out=None), hr.HR_ERR_INVALID_ARG), (dict(pos=None), hr.HR_ERR_INVALID_ARG),
    (dict(scales=None), hr.HR_ERR_INVALID_ARG), (dict(scales_out=None), hr.HR_ERR_INVALID_ARG),
    (dict(scales_width=0), hr.HR_ERR_INVALID_ARG), (dict(offsets=None), hr.HR_ERR_INVALID_ARG),
    (dict(experts=0), hr.HR_ERR_INVALID_ARG),
    (dict(in_stride=1023), hr.HR_ERR_INVALID_ARG), (dict(out_stride=1000), hr.HR_ERR_INVALID_ARG),
    (dict(scales_stride=7), hr.HR_ERR_INVALID_ARG), (dict(scales_out_stride=7), hr.HR_ERR_INVALID_ARG),
    (dict(tokens=0), hr.HR_OK), (dict(rows=0), hr.HR_OK),
    (dict(tokens=1 << 30), hr.HR_ERR_TOO_LARGE), (dict(rows=1 << 31), hr.HR_ERR_TOO_LARGE),
    (dict(row_bytes=1 << 31), hr.HR_ERR_TOO_LARGE),
    (dict(tokens=1 << 27, row_bytes=1024, out=at(4000), scales_out=at(9000), pos=at(10000), order=at(11000),
          offsets=at(11001), scales=at(12000)), hr.HR_ERR_TOO_LARGE),
    (dict(pos=at(4) + 2), hr.HR_ERR_ALIGNMENT), (dict(scales=at(1) + 2), hr.HR_ERR_ALIGNMENT),
    (dict(out=at(0)), hr.HR_ERR_INVALID_ARG), (dict(out=at(4) + 64), hr.HR_ERR_INVALID_ARG),
    (dict(scales_out=at(1)), hr.HR_ERR_INVALID_ARG), (dict(scales_out=at(2) + 4096), hr.HR_ERR_INVALID_ARG),
    (dict(out=at(5) + 4), hr.HR_ERR_INVALID_ARG)])
def test_gather_refusals(over, status):
    assert gather(**over) == status


def both(args, f16, bf16):
    got = {f16(args, 0), bf16(args, 0)}
    assert len(got) == 1
    return got.pop()


def combine(**over):
    a = hr.hr_experts_combine_args()
    a.z, a.addend, a.out, a.pos, a.weights = (at(i) for i in range(5))
    a.tokens, a.rows, a.hidden, a.k = 100, 400, 512, 4
    for n, v in over.items():
        setattr(a, n, v)
    return both(a, hr.hr_experts_combine_f16, hr.hr_experts_combine_bf16)


@pytest.mark.parametrize("over,status", [
    (dict(hidden=0), hr.HR_ERR_INVALID_ARG), (dict(k=0), hr.HR_ERR_INVALID_ARG), (dict(k=33), hr.HR_ERR_INVALID_ARG),
    (dict(z=None), hr.HR_ERR_INVALID_ARG), (dict(out=None), hr.HR_ERR_INVALID_ARG),
    (dict(pos=None), hr.HR_ERR_INVALID_ARG), (dict(tokens=0), hr.HR_OK),
    (dict(tokens=1 << 30), hr.HR_ERR_TOO_LARGE), (dict(rows=1 << 31), hr.HR_ERR_TOO_LARGE),
    (dict(hidden=1 << 27), hr.HR_ERR_TOO_LARGE),
    (dict(z_stride=511), hr.HR_ERR_INVALID_ARG), (dict(out_stride=511), hr.HR_ERR_INVALID_ARG),
    (dict(addend_stride=511), hr.HR_ERR_INVALID_ARG),
    (dict(z=at(0) + 1), hr.HR_ERR_ALIGNMENT), (dict(out=at(2) + 1), hr.HR_ERR_ALIGNMENT),
    (dict(weights=at(4) + 2), hr.HR_ERR_ALIGNMENT), (dict(pos=at(3) + 2), hr.HR_ERR_ALIGNMENT),
    (dict(out=at(0)), hr.HR_ERR_INVALID_ARG), (dict(out=at(1) + 2), hr.HR_ERR_INVALID_ARG),
    (dict(out=at(1), out_stride=1024), hr.HR_ERR_INVALID_ARG), (dict(out=at(3)), hr.HR_ERR_INVALID_ARG),
    (dict(out=at(4) - 2), hr.HR_ERR_INVALID_ARG)])
def test_combine_refusals(over, status):
    assert combine(**over) == status


def grad(**over):
    a = hr.hr_experts_combine_grad_args()
    a.dy, a.z, a.dz, a.pos, a.weights, a.dweights, a.order, a.offsets = (at(i) for i in range(8))
    a.tokens, a.rows, a.hidden, a.k, a.experts = 100, 400, 512, 4, 16
    for n, v in over.items():
        setattr(a, n, v)
    return both(a, hr.hr_experts_combine_grad_f16, hr.hr_experts_combine_grad_bf16)


@pytest.mark.parametrize("over,status", [
    (dict(hidden=0), hr.HR_ERR_INVALID_ARG), (dict(k=0), hr.HR_ERR_INVALID_ARG),
    (dict(dz=None, dweights=None), hr.HR_ERR_INVALID_ARG), (dict(dy=None), hr.HR_ERR_INVALID_ARG),
    (dict(z=None), hr.HR_ERR_INVALID_ARG), (dict(pos=None), hr.HR_ERR_INVALID_ARG),
    (dict(offsets=None), hr.HR_ERR_INVALID_ARG), (dict(experts=0), hr.HR_ERR_INVALID_ARG),
    (dict(tokens=0), hr.HR_OK), (dict(tokens=1 << 30), hr.HR_ERR_TOO_LARGE),
    (dict(dy_stride=511), hr.HR_ERR_INVALID_ARG), (dict(z_stride=511), hr.HR_ERR_INVALID_ARG),
    (dict(dz_stride=511), hr.HR_ERR_INVALID_ARG),
    (dict(dz=at(2) + 1), hr.HR_ERR_ALIGNMENT), (dict(dweights=at(5) + 2), hr.HR_ERR_ALIGNMENT),
    (dict(dz=at(0)), hr.HR_ERR_INVALID_ARG), (dict(dz=at(1) + 16), hr.HR_ERR_INVALID_ARG),
    (dict(dweights=at(4)), hr.HR_ERR_INVALID_ARG), (dict(dweights=at(1) + 64), hr.HR_ERR_INVALID_ARG),
    (dict(dweights=at(2) + 64), hr.HR_ERR_INVALID_ARG), (dict(dz=at(6) + 64), hr.HR_ERR_INVALID_ARG)])
def test_grad_refusals(over, status):
    assert grad(**over) == status


@pytest.mark.parametrize("tokens,k,experts,pad", [
    (5, hr.HR_EXPERTS_MAX_K + 1, 8, 1), (5, 1, hr.HR_EXPERTS_MAX + 1, 1), (1 << 31, 1, 8, 1), (1 << 26, 32, 8, 1),
    (2000, 8, 64, 1 << 30), ((1 << 31) - 1, 1, 8, 2)])
def test_sizes_of_what_a_sort_refuses(tokens, k, experts, pad):
    """No size for a call that hr_experts_sort refuses whatever the buffers."""
    assert sort(tokens=tokens, k=k, experts=experts, pad=pad, offsets=at(100), order=at(200), pos=at(300), ws=at(400),
                ws_bytes=1 << 60, rows=(1 << 31) - 1) == hr.HR_ERR_TOO_LARGE
    assert hr.hr_experts_rows(tokens, k, experts, pad) == 0
    if pad == 1:
        assert hr.hr_experts_sort_workspace(tokens, k, experts) == 0


def test_largest_sizes():
    assert hr.hr_experts_rows(5, hr.HR_EXPERTS_MAX_K, hr.HR_EXPERTS_MAX, 1) == 5 * hr.HR_EXPERTS_MAX_K
    assert hr.hr_experts_rows((1 << 31) - 1, 1, 8, 1) == (1 << 31) - 1
    assert hr.hr_experts_rows((1 << 31) - 1 - 8 * 15, 1, 8, 16) == (1 << 31) - 1
    assert hr.hr_experts_rows((1 << 31) - 8 * 15, 1, 8, 16) == 0
    assert hr.hr_experts_sort_workspace((1 << 31) - 1, 1, 8) > 0
    assert hr.hr_experts_sort_workspace(1 << 20, hr.HR_EXPERTS_MAX_K, hr.HR_EXPERTS_MAX) > 0
