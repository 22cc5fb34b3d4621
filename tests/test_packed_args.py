"""The operators around the combine pack their argument structs as bytes; here
the bytes of a call are read back as the C struct, field by field (CPU: the
library's function is replaced by one that keeps its argument), and the structs'
fields are compared with the header's."""
import ctypes
import os
import subprocess

import pytest
import torch

from message_fp16_all_amd import hr

F8 = torch.float8_e4m3fn


class Rows(torch.Tensor):
    """Host memory that takes itself for a device tensor; no kernel sees it."""
    is_cuda = property(lambda self: True)


class Stream:
    cuda_stream = 0xABC0


def rows(n, width, stride, dtype=torch.float16):
    return torch.zeros(n * stride, dtype=dtype).as_strided((n, width), (stride, 1)).as_subclass(Rows)


def flat(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Rows)


@pytest.fixture
def call(monkeypatch):
    """call(struct, entry point, function, ...) -> the struct that the function passed."""
    real = hr.load()

    def run(struct, entry, fn, *args, **kw):
        kept = []

        class Library:
            def __getattr__(self, name):
                return getattr(real, name)

        def keep(packed, stream):
            assert stream == Stream.cuda_stream
            kept.append(packed)
            return hr.HR_OK

        lib = Library()
        setattr(lib, entry, keep)
        monkeypatch.setattr(hr, "load", lambda: lib)
        monkeypatch.setattr(hr, "_entries", {})
        fn(*args, stream=Stream, **kw)
        assert len(kept) == 1 and len(kept[0]) == ctypes.sizeof(struct)
        return struct.from_buffer_copy(kept[0])

    return run


def check(got, **want):
    """Every field of the struct: tensors by their address, None as null."""
    assert {n for n, _ in got._fields_} == set(want)
    for name, value in want.items():
        field = [p or 0 for p in got.inputs] if name == "inputs" else getattr(got, name)
        if isinstance(value, torch.Tensor):
            value = value.data_ptr()
        assert (field or 0) == (value or 0), name


@pytest.mark.parametrize("dt,end", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
def test_norm(call, dt, end):
    n, w = 5, 256
    xs = [rows(n, w, 300, dt) for _ in range(3)]
    r, h, y = (rows(n, w, s, dt) for s in (310, 320, 330))
    codes, scales, rstd, weight = rows(n, w, 340, F8), rows(n, 8, 9, torch.float32), flat(n), flat(w)
    got = call(hr.hr_rmsnorm_args, f"hr_reduce_rmsnorm_{end}", hr.reduce_rmsnorm, xs, y, residual=r, residual_out=h,
               weight=weight, eps=0.5, out8=codes, scales=scales, group=32, rstd=rstd)
    check(got, inputs=[x.data_ptr() for x in xs] + [0] * (hr.HR_MAX_G - 3), residual=r, weight=weight,
          residual_out=h, out=y, codes=codes, scales=scales, rstd=rstd, rows=n, hidden=w, input_stride=300,
          residual_stride=310, residual_out_stride=320, out_stride=330, codes_stride=340, scales_stride=9, G=3,
          weight_f32=1, group=32, eps=0.5)
    got = call(hr.hr_rmsnorm_args, f"hr_reduce_rmsnorm_{end}", hr.reduce_rmsnorm, xs[:1], y)
    check(got, inputs=[xs[0].data_ptr()] + [0] * (hr.HR_MAX_G - 1), residual=None, weight=None,
          residual_out=None, out=y, codes=None, scales=None, rstd=None, rows=n, hidden=w, input_stride=300,
          residual_stride=0, residual_out_stride=0, out_stride=330, codes_stride=0, scales_stride=0, G=1, weight_f32=0,
          group=0, eps=got.eps)


@pytest.mark.parametrize("dt,end", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
def test_norm_grad(call, dt, end):
    n, w = 6, 128
    dy, h, r, dx = (rows(n, w, s, dt) for s in (130, 140, 150, 160))
    rstd, weight, dweight, ws = flat(n), flat(w), flat(w), flat(999, dtype=torch.uint8)
    got = call(hr.hr_rmsnorm_grad_args, f"hr_rmsnorm_grad_{end}", hr.rmsnorm_grad, dy, h, rstd, dx, weight=weight,
               dresidual=r, dweight=dweight, workspace=ws)
    check(got, dy=dy, h=h, rstd=rstd, weight=weight, dresidual=r, dx=dx, dweight=dweight, workspace=ws,
          workspace_bytes=999, rows=n, hidden=w, dy_stride=130, h_stride=140, dresidual_stride=150, dx_stride=160,
          weight_f32=1)


def test_gather(call):
    tokens, k, n, w = 4, 3, 20, 64
    x, out = rows(tokens, w, 70), rows(n, w, 80)
    s, so = rows(tokens, 2, 3, torch.float32), rows(n, 2, 5, torch.float32)
    pos, order, offsets = (flat(*shape, dtype=torch.int32) for shape in ((tokens, k), (n,), (8,)))
    got = call(hr.hr_experts_gather_args, "hr_experts_gather", hr.experts_gather, x, pos, out, offsets=offsets,
               order=order, scales=s, scales_out=so)
    check(got, in_=x, scales=s, out=out, scales_out=so, pos=pos, order=order, offsets=offsets, tokens=tokens, rows=n,
          row_bytes=2 * w, in_stride=140, out_stride=160, scales_width=2, scales_stride=3, scales_out_stride=5, k=k,
          experts=7)


@pytest.mark.parametrize("dt,end", [(torch.float16, "f16"), (torch.bfloat16, "bf16")])
def test_combine_and_its_gradient(call, dt, end):
    tokens, k, n, w = 4, 3, 20, 64
    z, add, out, dz = rows(n, w, 70, dt), rows(tokens, w, 80, dt), rows(tokens, w, 90, dt), rows(n, w, 100, dt)
    weights, dweights = flat(tokens, k), flat(tokens, k)
    pos, order, offsets = (flat(*shape, dtype=torch.int32) for shape in ((tokens, k), (n,), (8,)))
    got = call(hr.hr_experts_combine_args, f"hr_experts_combine_{end}", hr.experts_combine, z, pos, out,
               weights=weights, addend=add)
    check(got, z=z, addend=add, out=out, pos=pos, weights=weights, tokens=tokens, rows=n, hidden=w, z_stride=70,
          addend_stride=80, out_stride=90, k=k)
    got = call(hr.hr_experts_combine_grad_args, f"hr_experts_combine_grad_{end}", hr.experts_combine_grad, out, z, pos,
               weights, dz, dweights, offsets=offsets, order=order)
    check(got, dy=out, z=z, dz=dz, pos=pos, weights=weights, dweights=dweights, order=order, offsets=offsets,
          tokens=tokens, rows=n, hidden=w, dy_stride=90, z_stride=70, dz_stride=100, k=k, experts=7)


STRUCTS = (hr.hr_rmsnorm_args, hr.hr_rmsnorm_grad_args, hr.hr_experts_gather_args, hr.hr_experts_combine_args,
           hr.hr_experts_combine_grad_args)


def test_structs_are_the_headers(tmp_path):
    """Every field lies where a C compiler puts it."""
    fields = [(c, n) for c in STRUCTS for n, _ in c._fields_]
    lines = ["#include <stdio.h>", '#include "hr.h"', "int main(void) {"]
    for c, n in fields:
        f = n.rstrip("_")
        lines.append(f'printf("%zu %zu\\n", offsetof({c.__name__}, {f}), sizeof((({c.__name__} *)0)->{f}));')
    source = tmp_path / "fields.c"
    source.write_text("\n".join([*lines, "return 0;", "}", ""]))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-I", include, str(source), "-o", str(tmp_path / "fields")], check=True)
    out = subprocess.run([str(tmp_path / "fields")], check=True, capture_output=True, text=True).stdout.split("\n")
    assert len(out) == len(fields) + 1
    for (c, n), line in zip(fields, out):
        d = getattr(c, n)
        assert line == f"{d.offset} {d.size}", f"{c.__name__}.{n}"
