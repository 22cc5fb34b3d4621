"""The experts' products, their gradient and the activation refuse bad arguments
before any device call (CPU): the addresses below are never dereferenced.  Their
argument structs, read back from what the binding packs, and compared with the
header's."""
import ctypes
import os
import subprocess

import pytest
import torch

from message_fp16_all_amd import hr
from test_packed_args import call, check, flat, rows  # noqa: F401  (call is a fixture)

F8 = torch.float8_e4m3fn
BASE = 0x7F0000000000
STEP = 1 << 30
BAD, LARGE, ALIGN = hr.HR_ERR_INVALID_ARG, hr.HR_ERR_TOO_LARGE, hr.HR_ERR_ALIGNMENT


def at(i):
    return BASE + i * STEP


def both(args, f16, bf16):
    got = {f16(args, 0), bf16(args, 0)}
    assert len(got) == 1
    return got.pop()


def product(eight=False, **over):
    a = hr.hr_experts_product_args()
    a.x, a.w, a.out, a.offsets = (at(i) for i in range(4))
    if eight:
        a.x_scales, a.w_scales = at(4), at(5)
    a.rows, a.n, a.k, a.experts = 100, 384, 512, 8
    for n, v in over.items():
        setattr(a, n, v)
    return both(a, *((hr.hr_experts_product_e4m3_f16, hr.hr_experts_product_e4m3_bf16) if eight else
                     (hr.hr_experts_product_f16, hr.hr_experts_product_bf16)))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("over,status", [
    (dict(n=0), BAD), (dict(k=0), BAD), (dict(experts=0), BAD), (dict(experts=-1), BAD), (dict(offsets=None), BAD),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(out=None), BAD),
    (dict(n=(1 << 20) + 1), LARGE), (dict(k=(1 << 20) + 1), LARGE), (dict(experts=1025), LARGE), (dict(rows=1 << 31), LARGE),
    (dict(x_stride=511), BAD), (dict(out_stride=383), BAD), (dict(w_stride=511), BAD), (dict(w_expert_stride=383 * 512), BAD),
    (dict(transposed=1, w_stride=383), BAD), (dict(transposed=1, w_expert_stride=511 * 384), BAD),
    (dict(x_stride=(1 << 22) + 16), LARGE), (dict(w_stride=(1 << 22) + 16), LARGE), (dict(out_stride=(1 << 21) + 8), LARGE),
    (dict(x_stride=1 << 62), BAD), (dict(w_expert_stride=1 << 62), BAD),
    (dict(out=at(2) + 1), ALIGN), (dict(offsets=at(3) + 2), ALIGN),
    (dict(out=at(0)), BAD), (dict(out=at(0) + 100 * 512 - 2), BAD), (dict(out=at(1) + 64), BAD), (dict(out=at(3) + 32), BAD),
    (dict(rows=0), hr.HR_OK), (dict(rows=0, x=None, out=None), hr.HR_OK), (dict(rows=0, k=0), BAD)])
def test_product_refusals(eight, over, status):
    assert product(eight, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(x=at(0) + 1), ALIGN), (dict(w=at(1) + 1), ALIGN), (dict(x_scales=at(4)), BAD), (dict(w_scales=at(5)), BAD)])
def test_product_refusals_16(over, status):
    assert product(**over) == status


@pytest.mark.parametrize("over,status", [
    (dict(x_scales=None), BAD), (dict(w_scales=None), BAD), (dict(x_scales=at(4) + 2), ALIGN), (dict(w_scales=at(5) + 2), ALIGN),
    (dict(x_scales_stride=3), BAD), (dict(w_scales_stride=3), BAD), (dict(w_scales_expert_stride=11), BAD),
    (dict(transposed=1, w_scales_stride=2), BAD), (dict(out=at(4) + 64), BAD), (dict(out=at(5) + 8 * 12 * 4 - 4), BAD)])
def test_product_refusals_8(over, status):
    assert product(True, **over) == status


@pytest.mark.parametrize("eight", [False, True])
def test_most_rows(eight):
    """A row number plus a tile's or a stage's rows stays in 31 bits."""
    assert product(eight, rows=(1 << 31) - 4095) == LARGE
    assert product(eight, rows=(1 << 31) - 4096, out=at(2) + 1) == ALIGN
    assert grad(rows=(1 << 31) - 4095) == LARGE
    assert grad(rows=(1 << 31) - 4096, dw=at(2) + 1) == ALIGN


@pytest.mark.parametrize("eight", [False, True])
def test_one_row_is_not_apart_from_another(eight):
    """The distance of a row that no second one follows is not limited."""
    far, late = 1 << 30, dict(out=at(2) + 1)                     # (refused by what is looked at next)
    one = dict(rows=1, x_stride=far, out_stride=far, **(dict(x_scales_stride=far) if eight else {}))
    assert product(eight, **one, **late) == ALIGN
    assert product(eight, n=1, w_stride=far, **late) == ALIGN
    assert product(eight, k=1, transposed=1, w_stride=far, n=384, **late) == ALIGN
    assert product(eight, **{**one, "rows": 2}, **late) == LARGE
    assert product(eight, n=2, w_stride=far, **late) == LARGE
    assert product(eight, x_stride=far, rows=0) == hr.HR_OK
    late = dict(dw=at(2) + 1)
    assert grad(rows=1, dy_stride=far, x_stride=far, **late) == ALIGN
    assert grad(n=1, dw_stride=far, **late) == ALIGN
    assert grad(n=2, dw_stride=far, **late) == LARGE


def test_matrices_in_pieces():
    """The bytes between matrices that are apart are not theirs."""
    gap = dict(n=64, k=64, w_expert_stride=1 << 20)
    assert product(**gap, out=at(1) + 64 * 64 * 2 - 2) == BAD
    assert product(**gap, out=at(1) + (1 << 21) * 7 + 64 * 64 * 2 - 2) == BAD


def grad(**over):
    a = hr.hr_experts_product_grad_args()
    a.dy, a.x, a.dw, a.offsets = (at(i) for i in range(4))
    a.rows, a.n, a.k, a.experts = 100, 384, 512, 8
    for n, v in over.items():
        setattr(a, n, v)
    return both(a, hr.hr_experts_product_grad_f16, hr.hr_experts_product_grad_bf16)


@pytest.mark.parametrize("over,status", [
    (dict(n=0), BAD), (dict(k=0), BAD), (dict(experts=0), BAD), (dict(offsets=None), BAD), (dict(dw=None), BAD),
    (dict(dy=None), BAD), (dict(x=None), BAD), (dict(dw=None, rows=0), BAD),
    (dict(n=(1 << 20) + 1), LARGE), (dict(k=(1 << 20) + 1), LARGE), (dict(experts=1025), LARGE), (dict(rows=1 << 31), LARGE),
    (dict(dy_stride=383), BAD), (dict(x_stride=511), BAD), (dict(dw_stride=511), BAD), (dict(dw_expert_stride=512 * 383), BAD),
    (dict(dy_stride=(1 << 21) + 8), LARGE), (dict(dw_stride=(1 << 21) + 8), LARGE),
    (dict(dw_f32=1, dw_stride=(1 << 20) + 8), LARGE),
    (dict(dy=at(0) + 1), ALIGN), (dict(x=at(1) + 1), ALIGN), (dict(dw=at(2) + 1), ALIGN), (dict(dw_f32=1, dw=at(2) + 2), ALIGN),
    (dict(offsets=at(3) + 1), ALIGN),
    (dict(dw=at(0) + 2), BAD), (dict(dw=at(1) + 100 * 512 * 2 - 2), BAD), (dict(dw=at(3) - 8 * 384 * 512 * 2 + 2), BAD)])
def test_grad_refusals(over, status):
    assert grad(**over) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no kernel can start")
def test_largest_gradient():
    """Up to 2^32 work-items: of 128 x 128 values 2^24 tiles for all matrices together."""
    one = dict(rows=1, experts=1, offsets=None)
    odd = dict(k=(1 << 18) + 1)
    assert grad(**one, n=(1 << 17) + 1, **odd) == hr.HR_ERR_HIP
    assert grad(**one, n=(1 << 18) + 1, **odd) == hr.HR_ERR_HIP          # 2^22 tiles and more
    assert grad(**one, n=8187 * 128, **odd) == hr.HR_ERR_HIP
    assert grad(**one, n=8187 * 128 + 1, **odd) == LARGE
    assert grad(rows=1, offsets=BASE - STEP, n=(1 << 18) + 1, **odd) == LARGE      # eight of them


def act(**over):
    a = hr.hr_experts_act_args()
    a.x, a.out, a.codes, a.scales, a.offsets = (at(i) for i in range(5))
    a.rows, a.width, a.gated, a.group, a.experts = 100, 384, 1, 128, 8
    for n, v in over.items():
        setattr(a, n, v)
    return both(a, hr.hr_experts_act_f16, hr.hr_experts_act_bf16)


@pytest.mark.parametrize("over,status", [
    (dict(width=0), BAD), (dict(group=0), BAD), (dict(group=16), BAD), (dict(group=256), BAD), (dict(experts=0), BAD),
    (dict(codes=None), BAD), (dict(scales=None), BAD), (dict(x=None), BAD), (dict(out=None, codes=None, scales=None), BAD),
    (dict(rows=1 << 31), LARGE), (dict(width=(1 << 20) + 1), LARGE),
    (dict(x_stride=767), BAD), (dict(out_stride=383), BAD), (dict(codes_stride=383), BAD), (dict(scales_stride=2), BAD),
    (dict(x=at(0) + 1), ALIGN), (dict(out=at(1) + 1), ALIGN), (dict(scales=at(3) + 2), ALIGN), (dict(offsets=at(4) + 2), ALIGN),
    (dict(out=at(0)), BAD), (dict(codes=at(0) + 100 * 768 * 2 - 1), BAD), (dict(scales=at(1) + 64), BAD),
    (dict(codes=at(1) + 5), BAD), (dict(out=at(4) + 8), BAD), (dict(scales=at(4) + 32), BAD), (dict(scales=at(2) + 4), BAD),
    (dict(rows=0), hr.HR_OK), (dict(rows=0, x=None), hr.HR_OK)])
def test_act_refusals(over, status):
    assert act(**over) == status


def act_grad(**over):
    a = hr.hr_experts_act_grad_args()
    a.dy, a.x, a.dx, a.out, a.offsets = (at(i) for i in range(5))
    a.rows, a.width, a.experts = 100, 384, 8
    for n, v in over.items():
        setattr(a, n, v)
    return both(a, hr.hr_experts_act_grad_f16, hr.hr_experts_act_grad_bf16)


@pytest.mark.parametrize("over,status", [
    (dict(width=0), BAD), (dict(experts=0), BAD), (dict(dy=None), BAD), (dict(x=None), BAD), (dict(dx=None), BAD),
    (dict(rows=1 << 31), LARGE), (dict(width=(1 << 20) + 1), LARGE),
    (dict(dy_stride=383), BAD), (dict(x_stride=767), BAD), (dict(dx_stride=767), BAD), (dict(out_stride=383), BAD),
    (dict(dy=at(0) + 1), ALIGN), (dict(dx=at(2) + 1), ALIGN), (dict(out=at(3) + 1), ALIGN), (dict(offsets=at(4) + 1), ALIGN),
    (dict(dx=at(1), dx_stride=1000), BAD), (dict(dx=at(1) + 2), BAD), (dict(dx=at(0)), BAD), (dict(out=at(0)), BAD),
    (dict(out=at(1)), BAD), (dict(out=at(2) + 768), BAD), (dict(dx=at(4) + 4), BAD), (dict(out=at(4) + 4), BAD),
    (dict(rows=0), hr.HR_OK)])
def test_act_grad_refusals(over, status):
    assert act_grad(**over) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where no kernel can start")
@pytest.mark.parametrize("width,most", [(513, (1 << 25) - 2), (1 << 20, (1 << 25) - 2), (512, (1 << 27) - 8),
                                        (129, (1 << 27) - 8), (128, (1 << 29) - 32), (1, (1 << 29) - 32)])
def test_most_rows_of_the_activation(width, most):
    """A launch has fewer than 2^32 work-items: the rows that the header names."""
    far = [(i + 1) << 56 for i in range(4)]                      # (the buffers take up to 2^47 bytes)
    forward = dict(width=width, x=far[0], out=far[1], codes=None, scales=None, offsets=None, experts=0)
    back = dict(width=width, dy=far[0], x=far[1], dx=far[2], out=far[3], offsets=None, experts=0)
    for rows, status in ((most, hr.HR_ERR_HIP), (most + 1, LARGE), ((1 << 31) - 1, LARGE)):
        assert act(rows=rows, **forward) == status
        assert act(rows=rows, gated=0, **forward) == status
        assert act_grad(rows=rows, **back) == status


# ---------------------------------------------------------------- the binding

@pytest.mark.parametrize("dt,end", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
def test_packed_product(call, dt, end):
    n, k, w, e = 6, 48, 32, 3
    x, out = rows(n, k, 50, dt), rows(n, w, 40, dt)
    offsets = flat(e + 1, dtype=torch.int32)
    m = rows(e * 40, k, 56, dt).as_strided((e, w, k), (40 * 56, 56, 1))
    got = call(hr.hr_experts_product_args, f"hr_experts_product_{end}", hr.experts_product, x, m, out, offsets=offsets)
    check(got, x=x, w=m, out=out, offsets=offsets, x_scales=None, w_scales=None, rows=n, n=w, k=k, x_stride=50,
          out_stride=40, w_stride=56, w_expert_stride=40 * 56, x_scales_stride=0, w_scales_stride=0,
          w_scales_expert_stride=0, experts=e, transposed=0)
    y, back = rows(n, w, 40, dt), rows(n, k, 50, dt)
    got = call(hr.hr_experts_product_args, f"hr_experts_product_{end}", hr.experts_product, y, m, back, offsets=offsets,
               transposed=True)
    check(got, x=y, w=m, out=back, offsets=offsets, x_scales=None, w_scales=None, rows=n, n=k, k=w, x_stride=40,
          out_stride=50, w_stride=56, w_expert_stride=40 * 56, x_scales_stride=0, w_scales_stride=0,
          w_scales_expert_stride=0, experts=e, transposed=1)


@pytest.mark.parametrize("dt,end", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
def test_packed_product_8(call, dt, end):
    n, k, w, e = 6, 300, 200, 3
    x, out = rows(n, k, 310, torch.uint8).view(F8), rows(n, w, 210, dt)
    m = flat(e, w, k, dtype=torch.uint8).view(F8)
    ms = flat(e, 2, 3)
    offsets = flat(e + 1, dtype=torch.int32)
    xs = rows(n, 3, 5, torch.float32)
    got = call(hr.hr_experts_product_args, f"hr_experts_product_e4m3_{end}", hr.experts_product, x, m, out,
               offsets=offsets, x_scales=xs, w_scales=ms)
    check(got, x=x, w=m, out=out, offsets=offsets, x_scales=xs, w_scales=ms, rows=n, n=w, k=k, x_stride=310,
          out_stride=210, w_stride=k, w_expert_stride=w * k, x_scales_stride=5, w_scales_stride=3,
          w_scales_expert_stride=6, experts=e, transposed=0)
    got = call(hr.hr_experts_product_args, f"hr_experts_product_e4m3_{end}", hr.experts_product, x, m[0], out,
               x_scales=xs, w_scales=ms[0])
    check(got, x=x, w=m, out=out, offsets=None, x_scales=xs, w_scales=ms, rows=n, n=w, k=k, x_stride=310,
          out_stride=210, w_stride=k, w_expert_stride=0, x_scales_stride=5, w_scales_stride=3,
          w_scales_expert_stride=0, experts=1, transposed=0)


@pytest.mark.parametrize("dt,end", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
@pytest.mark.parametrize("f32", [False, True])
def test_packed_grad(call, dt, end, f32):
    n, k, w, e = 6, 48, 32, 3
    dy, x, dw = rows(n, w, 40, dt), rows(n, k, 50, dt), flat(e, w, k, dtype=torch.float32 if f32 else dt)
    offsets = flat(e + 1, dtype=torch.int32)
    got = call(hr.hr_experts_product_grad_args, f"hr_experts_product_grad_{end}", hr.experts_product_grad, dy, x, dw,
               offsets=offsets)
    check(got, dy=dy, x=x, dw=dw, offsets=offsets, rows=n, n=w, k=k, dy_stride=40, x_stride=50, dw_stride=k,
          dw_expert_stride=w * k, experts=e, dw_f32=int(f32))


@pytest.mark.parametrize("dt,end", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
def test_packed_act(call, dt, end):
    n, w, e = 5, 96, 7
    x, out, codes, scales = rows(n, 2 * w, 200, dt), rows(n, w, 100, dt), rows(n, w, 104, F8), rows(n, 3, 4, torch.float32)
    offsets = flat(e + 1, dtype=torch.int32)
    got = call(hr.hr_experts_act_args, f"hr_experts_act_{end}", hr.experts_act, x, out, offsets=offsets, out8=codes,
               scales=scales, group=32)
    check(got, x=x, out=out, codes=codes, scales=scales, offsets=offsets, rows=n, width=w, x_stride=200, out_stride=100,
          codes_stride=104, scales_stride=4, gated=1, group=32, experts=e)
    dy, dx = rows(n, w, 110, dt), rows(n, 2 * w, 210, dt)
    got = call(hr.hr_experts_act_grad_args, f"hr_experts_act_grad_{end}", hr.experts_act_grad, dy, x, dx, out=out,
               offsets=offsets)
    check(got, dy=dy, x=x, dx=dx, out=out, offsets=offsets, rows=n, width=w, dy_stride=110, x_stride=200, dx_stride=210,
          out_stride=100, experts=e)


def test_binding_refusals():
    x, out, w = rows(4, 64, 64), rows(4, 32, 32), flat(2, 32, 64, dtype=torch.float16)
    off = flat(3, dtype=torch.int32)
    bad = [
        (ValueError, lambda: hr.experts_product(x, w, out)),                                   # several, no offsets
        (ValueError, lambda: hr.experts_product(x, w, out, offsets=flat(4, dtype=torch.int32))),
        (ValueError, lambda: hr.experts_product(x, w, out, offsets=off, transposed=True)),
        (ValueError, lambda: hr.experts_product(x, w, rows(4, 31, 31), offsets=off)),
        (ValueError, lambda: hr.experts_product(x, w, rows(5, 32, 32), offsets=off)),
        (TypeError, lambda: hr.experts_product(x, w.float(), out, offsets=off)),
        (TypeError, lambda: hr.experts_product(x.float(), w, out.float(), offsets=off)),
        (TypeError, lambda: hr.experts_product(torch.zeros(4, 64).half(), w, out, offsets=off)),  # host memory
        (ValueError, lambda: hr.experts_product(x, w.transpose(1, 2), out, offsets=off)),
        (ValueError, lambda: hr.experts_product(x, w, out, offsets=off, x_scales=flat(4, 1))),
        (TypeError, lambda: hr.experts_product(x, w, out, offsets=off, x_scales=flat(4, 1), w_scales=flat(2, 1, 1))),
        (ValueError, lambda: hr.experts_product_grad(out, x[:3], w, offsets=off)),
        (ValueError, lambda: hr.experts_product_grad(x, out, w, offsets=off)),
        (TypeError, lambda: hr.experts_product_grad(out, x, w.bfloat16(), offsets=off)),
        (ValueError, lambda: hr.experts_act(rows(4, 63, 63), rows(4, 31, 31))),
        (ValueError, lambda: hr.experts_act(x, rows(4, 64, 64))),
        (ValueError, lambda: hr.experts_act(x, out, gated=False)),
        (ValueError, lambda: hr.experts_act(x, out8=rows(4, 32, 32, F8), scales=flat(4, 2))),
        (ValueError, lambda: hr.experts_act_grad(out, rows(4, 60, 60), x)),
    ]
    for i, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            pytest.fail(f"call {i} was taken")
    x8, w8 = rows(4, 256, 256, torch.uint8).view(F8), flat(2, 32, 256, dtype=torch.uint8).view(F8)
    with pytest.raises(ValueError):
        hr.experts_product(x8, w8, out, offsets=off, x_scales=flat(4, 3), w_scales=flat(2, 1, 2))
    with pytest.raises(ValueError):
        hr.experts_product(x8, w8, out, offsets=off, x_scales=flat(4, 2), w_scales=flat(2, 2, 1))


STRUCTS = (hr.hr_experts_product_args, hr.hr_experts_product_grad_args, hr.hr_experts_act_args,
           hr.hr_experts_act_grad_args)


def test_structs_are_the_headers(tmp_path):
    """Every field lies where a C compiler puts it, and the packed forms are as long."""
    fields = [(c, n) for c in STRUCTS for n, _ in c._fields_]
    lines = ["#include <stdio.h>", '#include "hr.h"', "int main(void) {"]
    lines += [f'printf("%zu %zu\\n", offsetof({c.__name__}, {n}), sizeof((({c.__name__} *)0)->{n}));' for c, n in fields]
    source = tmp_path / "fields.c"
    source.write_text("\n".join([*lines, "return 0;", "}", ""]))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-I", include, str(source), "-o", str(tmp_path / "fields")], check=True)
    out = subprocess.run([str(tmp_path / "fields")], check=True, capture_output=True, text=True).stdout.split("\n")
    assert len(out) == len(fields) + 1
    for (c, n), line in zip(fields, out):
        d = getattr(c, n)
        assert line == f"{d.offset} {d.size}", f"{c.__name__}.{n}"
    for c, p in zip(STRUCTS, (hr._PRODUCT, hr._PRODUCT_GRAD, hr._ACT, hr._ACT_GRAD)):
        assert ctypes.sizeof(c) == p.size
