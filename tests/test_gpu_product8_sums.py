"""GPU: what the sums of e4m3 products hold, as the header states it: eight products of
adjacent values are cut at 2^-13 of the largest one's leading bit, and everything
beyond them is binary32.
"""
import pytest
import torch

from _gpu import needs_gpu
from _products import F8, product_ref, sum_tol, wide_blocks, wide_rows
from _rows import Maker, within
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"


def product(x, w, transposed=False, xs=None, ws=None):
    (rows, k), n = x.shape, w.shape[1] if transposed else w.shape[0]
    out = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
    xs = torch.ones(rows, -(-k // 128)) if xs is None else xs
    ws = torch.ones(*(-(-v // 128) for v in w.shape)) if ws is None else ws
    hr.experts_product(x.to(DEV), w.to(DEV), out, transposed=transposed, x_scales=xs.to(DEV), w_scales=ws.to(DEV))
    return out.cpu()


# (rows, k, n): few rows, whose waves split k; large tiles; odd lengths
@pytest.mark.parametrize("rows,k,n", [(3, 256, 32), (52000, 256, 272), (3, 253, 33), (1000, 253, 2063)])
@pytest.mark.parametrize("transposed", [False, True])
def test_small_beside_large(rows, k, n, transposed):
    """256 - 256 and, in another eight, 2^-9: 17 bits below, which binary32 holds.  Every value is exact
    in the sums, so the result is too."""
    m = Maker(rows + k)
    big = torch.randint(0, k, (rows,), generator=m.g)
    other = (big + 8 * torch.randint(1, 16, (rows,), generator=m.g)) % (k // 8 * 8)
    small = torch.randint(0, k, (rows,), generator=m.g)
    r = torch.arange(rows)
    apart = (small // 8 != big // 8) & (small // 8 != other // 8) & (big // 8 != other // 8)
    assert apart.sum() > 0
    big, other, small, r = big[apart], other[apart], small[apart], r[apart]
    x = torch.zeros(rows, k)
    x[r, big], x[r, other], x[r, small] = 256.0, -256.0, 2.0 ** -9
    got = product(x.to(F8), torch.ones(*((k, n) if transposed else (n, k))).to(F8), transposed)
    want = torch.zeros(rows, n, dtype=torch.bfloat16)
    want[r] = 2.0 ** -9
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows,k,n", [(3, 256, 32), (100, 512, 272), (3600, 272, 3600), (70, 253, 331)])
@pytest.mark.parametrize("transposed", [False, True])
def test_values_of_every_size(rows, k, n, transposed):
    """Magnitudes spread over e4m3's whole range, from 2^-9 to 448, next to each other."""
    m = Maker(k + n)

    def spread(*shape):
        e = torch.randint(-9, 9, shape, generator=m.g).float()
        v = torch.exp2(e) * (1 + torch.randint(0, 8, shape, generator=m.g) / 8)
        return (v.clamp(max=448) * (2 * torch.randint(0, 2, shape, generator=m.g) - 1)).to(F8)

    x, w = spread(rows, k), spread(*((k, n) if transposed else (n, k)))
    xs = torch.exp2(m.normal(rows, -(-k // 128)).clamp(-4, 4))
    ws = torch.exp2(m.normal(*(-(-v // 128) for v in w.shape)).clamp(-4, 4))
    got = product(x, w, transposed, xs, ws)
    ref, mag = product_ref(wide_rows(x, xs), wide_blocks(w, ws)[None], [0, rows], transposed)
    within(got, ref, sum_tol(torch.bfloat16, ref, mag, k, eight=True), "out")
