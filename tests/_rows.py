"""Helpers shared by the tests of the row operators (norm, router, experts):
bits of either 16-bit type, buffers at odd addresses and strides, and the
bounds that outputs are held to.

Bounds.  A rounding to a type is off by at most half a step, finfo(t).eps / 2
of the value, or half the smallest subnormal.  A row's binary32 work (a sum
over at most 64 sequential additions per lane and a tree of 10, a square root,
a quotient, four products) is fewer than 2^7 roundings of 2^-24 each, hence
F32 = 2^-17 of the magnitudes that go into a value.
"""
import numpy as np
import torch

import oracle

F32 = 2.0 ** -17
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype, ref):
    """Half a step of ``dtype`` at ``ref`` (a float64 tensor)."""
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.tiny * fi.eps / 2


def bits(t):
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def fold_ref(ts):
    """The oracle's fold of 16-bit tensors, as a tensor of their type (CPU)."""
    dt = ts[0].dtype
    xs = [bits(t).reshape(-1) for t in ts]
    out = oracle.fold_bf16(xs) if dt is torch.bfloat16 else oracle.fold(xs)
    return torch.from_numpy(out.view(np.int16).copy()).view(dt).reshape(ts[0].shape)


def same(got, ref, what):
    """Bit equality, NaN by class."""
    a, b = bits(got), bits(ref)
    ok = oracle.same_bits_bf16(a.reshape(-1), b.reshape(-1)) if got.dtype is torch.bfloat16 else \
        oracle.same_bits(a.reshape(-1), b.reshape(-1))
    assert ok.all(), f"{what}: {np.count_nonzero(~ok)} of {ok.size} values differ"


def within(got, ref, tol, what):
    """|got - ref| <= tol where ref is finite; the same infinities and NaN elsewhere."""
    got = got.detach().double().cpu()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    other = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[other], ref[other]), f"{what}: infinities differ"
    d = (got - ref).abs()[fine]
    t = tol[fine]
    bad = ~(d <= t)
    if bad.any():
        j = int(torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; first "
                             f"{float(got[fine][j])!r} against {float(ref[fine][j])!r}, bound {float(t[j]):.3g}")


class Maker:
    """Device tensors of a seed; ``place`` puts rows at a stride and an offset
    of values, inside a buffer whose other values must stay what they were."""

    def __init__(self, seed, device="cuda:0"):
        self.g = torch.Generator().manual_seed(seed)
        self.dev = device
        self.frames = []

    def normal(self, *shape, sigma=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g) * sigma).to(dtype)

    def place(self, rows, width, dtype, stride=None, offset=0, values=None, fill=7.0):
        stride = width if stride is None else stride
        n = offset + max(0, rows - 1) * stride + width + 5
        buf = torch.full((n,), fill, dtype=torch.float32).to(dtype).to(self.dev)
        view = buf.as_strided((rows, width), (stride, 1), offset)
        if values is not None:
            view.copy_(values.to(self.dev))
        else:
            inside = torch.zeros(n, dtype=torch.bool)
            inside.as_strided((rows, width), (stride, 1), offset).fill_(True)
            self.frames.append((buf, inside, fill))
        return view

    def check_frames(self):
        """Nothing outside the outputs' rows was written."""
        for buf, inside, fill in self.frames:
            rest = buf.float().cpu()[~inside]
            want = torch.full_like(rest, float(torch.tensor(fill).to(buf.dtype).float()))
            assert torch.equal(rest, want), "written outside an output's rows"
