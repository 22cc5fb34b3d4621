"""References and bounds of the experts' products and activation.

Bounds.  An output is rounded once to its type (half a step).  Before that a sum
of n products in binary32 is off by at most n roundings of 2^-24 (a matrix
instruction's own additions included, each of which keeps binary32) of the
magnitudes added, which ``mag`` holds: the same sum over absolute values.  e4m3:
the instruction adds its products eight at a time, cutting each at 2^-13 of the
largest one's leading bit, so eight products lose at most 7 * 2^-13 of that and
2^-10 of their magnitudes covers it; two roundings of 2^-24 for the scales.
"""
import torch

from _rows import half_step

F8 = torch.float8_e4m3fn


def sum_tol(dtype, ref, mag, n, eight=False):
    tol = mag * (n + 4) * 2.0 ** -24
    if eight:
        tol = tol + mag * 2.0 ** -10
    # (rounding what is already off: half a step of a value that far away)
    return half_step(dtype, ref) + tol * (1 + torch.finfo(dtype).eps)


def bounds_of(offsets, rows):
    return [(e, a, b) for e, (a, b) in enumerate(zip(offsets, offsets[1:]))]


def product_ref(x, w, offsets, transposed):
    """(out, the same over magnitudes) in 64 bits of CPU tensors; rows of no
    segment are NaN."""
    n = w.shape[2] if transposed else w.shape[1]
    out = torch.full((x.shape[0], n), float("nan"), dtype=torch.float64)
    mag = torch.zeros_like(out)
    x, w = x.double(), w.double()
    for e, a, b in bounds_of(offsets, x.shape[0]):
        m = w[e] if transposed else w[e].t()
        out[a:b] = x[a:b] @ m
        mag[a:b] = x[a:b].abs() @ m.abs()
    return out, mag


def grad_ref(dy, x, offsets):
    E = len(offsets) - 1
    out = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    dy, x = dy.double(), x.double()
    for e, a, b in bounds_of(offsets, x.shape[0]):
        out[e] = dy[a:b].t() @ x[a:b]
        mag[e] = dy[a:b].abs().t() @ x[a:b].abs()
    return out, mag


def wide_rows(codes, scales):
    """What codes with a scale per 128 columns stand for, in 64 bits."""
    return codes.double() * scales.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]


def wide_blocks(codes, scales):
    """The same with a scale per 128 x 128."""
    s = scales.double().repeat_interleave(128, -2)[..., :codes.shape[-2], :]
    return codes.double() * s.repeat_interleave(128, -1)[..., :codes.shape[-1]]
