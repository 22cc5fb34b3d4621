"""GPU: the activation's value before it is rounded to 16 bits or 8.

A group that holds one value other than zero has the scale |y| / 448 in binary32,
which shows y to 24 bits.

Bound, in units of 2^-23 of the value.  z = e^-gate: the exponential's 1, what
correcting its exponent rounds off 1/2 (the correction's own error is below
2^-30); 1 + z 1/2; the reciprocal 1; two products 1/2 each; the scale's quotient
1/2: 4.5 in all.  (Of a gate of 87 or more in magnitude: no sum and a reciprocal
of 1; one product more: 4.)
"""
import pytest
import torch

from _gpu import needs_gpu
from _products import F8
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"
UNIT = 2.0 ** -23
GROUP = 32


def scales_of(gate, up):
    """The scale of each gate alone in a group of its own, and the formula's in 64 bits."""
    x = torch.zeros(gate.numel(), 2 * GROUP, dtype=gate.dtype)
    x[:, 5], x[:, GROUP + 5] = gate, up
    codes = torch.empty(gate.numel(), GROUP, dtype=F8, device=DEV)
    scales = torch.empty(gate.numel(), 1, device=DEV)
    hr.experts_act(x.to(DEV), out8=codes, scales=scales, group=GROUP)
    g = gate.double()
    return scales.cpu()[:, 0].double(), (g * torch.sigmoid(g) * up).abs() / 448.0


def check(gate, up):
    got, want = scales_of(gate, up)
    assert (want > 2.0 ** -125).all()                             # (above the smallest scale, normal)
    off = ((got - want).abs() / want / UNIT)
    worst = off.argmax()
    assert off[worst] <= 4.5 * (1 + 2.0 ** -20), f"gate {gate[worst].item()}: {off[worst].item():.2f} units"


@pytest.mark.parametrize("low,high", [(0, 5), (5, 20), (20, 60), (60, 87)])
@pytest.mark.parametrize("sign", [1, -1])
def test_every_near_gate_of_float16(low, high, sign):
    """Every float16 number up to 87, but those below 2^-14."""
    bits = torch.arange(0x0400, 0x7C00, dtype=torch.int16)
    v = bits.view(torch.float16)
    v = v[(v >= low) & (v < high)]
    check(v * sign, 1024.0)


@pytest.mark.parametrize("sign", [1, -1])
def test_near_gates_of_bfloat16(sign):
    bits = torch.arange(0x3800, 0x42AE, dtype=torch.int16)
    check(bits.view(torch.bfloat16) * sign, 2.0 ** 40)


@pytest.mark.parametrize("sign", [1, -1])
def test_far_gates_of_bfloat16(sign):
    """From 87 up to 128."""
    bits = torch.arange(0x42AE, 0x4301, dtype=torch.int16)
    check(bits.view(torch.bfloat16) * sign, 2.0 ** 100)


def test_near_gates_beside_far_ones():
    """A near gate's value has the same bits beside a gate that is not near."""
    gate = torch.linspace(-86, 86, 4001).to(torch.float16)
    alone, _ = scales_of(gate, 1024.0)
    mixed = torch.stack([gate, torch.full_like(gate, -100.0)], 1).view(-1)
    beside, _ = scales_of(mixed, 1024.0)
    assert torch.equal(beside[::2], alone)
