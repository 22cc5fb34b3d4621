"""GPU: the experts' products and the matrices' gradient against 64 bits."""
import pytest
import torch

from _gpu import needs_gpu
from _products import F8, grad_ref, product_ref, sum_tol, wide_blocks, wide_rows
from _rows import TYPES, Maker, within
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"


def offsets_of(counts, first=0):
    at = [first]
    for c in counts:
        at.append(at[-1] + c)
    return at


def on_device(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device=DEV)


def check_rows(m, got, ref, tol, offsets, what, before=7.0):
    """The segments' rows within the bound, every other row as it was."""
    got = got.cpu()
    inside = torch.zeros(got.shape[0], dtype=torch.bool)
    inside[offsets[0]:offsets[-1]] = True
    within(got[inside], ref[inside], tol[inside], what)
    assert (got[~inside].float() == before).all(), f"{what}: wrote rows of no segment"
    m.check_frames()


# (counts of the experts' rows, rows behind the last, k, n)
SHAPES = [
    ([1], 0, 1, 1), ([1], 0, 8, 8), ([3], 2, 16, 24), ([1], 0, 64, 64), ([2, 0, 1], 3, 128, 64), ([0, 0], 4, 64, 64),
    ([1, 1, 0, 2, 1], 0, 200, 72), ([17, 15, 16], 1, 72, 136), ([40, 33, 31, 0], 5, 136, 200), ([64, 63, 65], 0, 256, 128),
    ([100, 130, 0, 127, 129], 0, 192, 264), ([300], 7, 320, 520), ([255, 257], 0, 64, 256), ([600, 1, 0, 200], 9, 520, 272),
    ([5, 0, 9], 2, 7, 9), ([33, 1], 0, 65, 63), ([130, 7], 3, 129, 257), ([300, 5], 0, 77, 131), ([1], 0, 1001, 3),
]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,behind,k,n", SHAPES)
def test_product(name, transposed, counts, behind, k, n):
    dt, E = TYPES[name], len(counts)
    m = Maker(k * 1000 + n)
    offsets = offsets_of(counts)
    rows = offsets[-1] + behind
    x, w = m.normal(rows, k, dtype=dt), m.normal(E, *((k, n) if transposed else (n, k)), dtype=dt)
    out = m.place(rows, n, dt)
    hr.experts_product(x.to(DEV), w.to(DEV), out, offsets=on_device(offsets), transposed=transposed)
    ref, mag = product_ref(x, w, offsets, transposed)
    check_rows(m, out, ref, sum_tol(dt, ref, mag, k), offsets, "out")


def eight(m, rows, width, blocks=False):
    """Codes over the whole range, scales of several sizes."""
    codes = (m.normal(rows, width, sigma=100.0)).clamp(-448, 448).to(F8)
    r = -(-rows // 128) if blocks else rows
    scales = torch.exp2(m.normal(r, -(-width // 128)).clamp(-3, 3))
    return codes, scales


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,behind,k,n", SHAPES)
def test_product8(name, transposed, counts, behind, k, n):
    dt, E = TYPES[name], len(counts)
    m = Maker(k * 1000 + n + 1)
    offsets = offsets_of(counts)
    rows = offsets[-1] + behind
    x, xs = eight(m, rows, k)
    xs = xs * 2.0 ** -8                                          # (float16 sums stay finite)
    ws = [eight(m, *((k, n) if transposed else (n, k)), blocks=True) for _ in range(E)]
    w, wsc = torch.stack([a.view(torch.uint8) for a, _ in ws]).view(F8), torch.stack([b for _, b in ws]) * 2.0 ** -8
    out = m.place(rows, n, dt)
    hr.experts_product(x.to(DEV), w.to(DEV), out, offsets=on_device(offsets), transposed=transposed,
                       x_scales=xs.to(DEV), w_scales=wsc.to(DEV))
    ref, mag = product_ref(wide_rows(x, xs), wide_blocks(w, wsc), offsets, transposed)
    check_rows(m, out, ref, sum_tol(dt, ref, mag, k, eight=True), offsets, "out")


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts,behind,k,n", SHAPES)
def test_product_grad(name, f32, counts, behind, k, n):
    dt, E = TYPES[name], len(counts)
    m = Maker(k * 1000 + n + 2)
    offsets = offsets_of(counts)
    rows = offsets[-1] + behind
    dy, x = m.normal(rows, n, dtype=dt), m.normal(rows, k, dtype=dt)
    # what no expert owns may be anything
    dy[offsets[-1]:], x[offsets[-1]:] = float("nan"), float("inf")
    to = torch.float32 if f32 else dt
    dw = m.place(E * n, k, to).view(E, n, k)
    hr.experts_product_grad(dy.to(DEV), x.to(DEV), dw, offsets=on_device(offsets))
    ref, mag = grad_ref(dy, x, offsets)
    within(dw.cpu(), ref, sum_tol(to, ref, mag, max(counts)), "dw")
    m.check_frames()


def many(seed, experts=48, pad=1):
    """Offsets of segments of every height up to three tiles, more tiles than the GPU has compute units."""
    g = torch.Generator().manual_seed(seed)
    counts = (torch.randint(0, 640, (experts,), generator=g) + pad - 1) // pad * pad
    counts[3], counts[4], counts[5], counts[6], counts[7] = 0, 128, 256, 384, 512
    return offsets_of(counts.tolist())


def rows_ref(x, w, offsets, transposed):
    """product_ref in 64 bits on the GPU, a segment at a time."""
    n = w.shape[2] if transposed else w.shape[1]
    out = torch.full((x.shape[0], n), float("nan"), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        xs, m = x[a:b].to(DEV).double(), w[e].to(DEV).double()
        m = m if transposed else m.t()
        out[a:b], mag[a:b] = (xs @ m).cpu(), (xs.abs() @ m.abs()).cpu()
    return out, mag


@pytest.mark.parametrize("k,n,transposed", [(64, 1024, False), (72, 1288, True), (328, 1016, False), (192, 1100, True),
                                            (128, 1024, True), (520, 1032, False)])
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
def test_many_tiles(kind, k, n, transposed):
    """Workgroups that compute several tiles, whole and partial ones in turn."""
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    m = Maker(k + n)
    offsets = many(k)
    rows, E = offsets[-1] + 3, len(offsets) - 1
    if kind == "e4m3":
        k, n = k // 16 * 16, n // 16 * 16
        x, xs = eight(m, rows, k)
        ws = [eight(m, *((k, n) if transposed else (n, k)), blocks=True) for _ in range(E)]
        w, wsc = torch.stack([a.view(torch.uint8) for a, _ in ws]).view(F8), torch.stack([b for _, b in ws]) * 2.0 ** -8
        scales = dict(x_scales=xs.to(DEV), w_scales=wsc.to(DEV))
        xw, ww = wide_rows(x, xs), wide_blocks(w, wsc)
    else:
        x, w = m.normal(rows, k, dtype=dt), m.normal(E, *((k, n) if transposed else (n, k)), dtype=dt)
        scales, xw, ww = {}, x, w
    out = m.place(rows, n, dt)
    hr.experts_product(x.to(DEV), w.to(DEV), out, offsets=on_device(offsets), transposed=transposed, **scales)
    ref, mag = rows_ref(xw, ww, offsets, transposed)
    check_rows(m, out, ref, sum_tol(dt, ref, mag, k, eight=kind == "e4m3"), offsets, "out")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("k,n", [(512, 512), (520, 392), (264, 1000)])
def test_many_tiles_grad(name, f32, k, n):
    dt = TYPES[name]
    m = Maker(k * n)
    offsets = many(k + 1, experts=100)
    rows, E = offsets[-1], len(offsets) - 1
    dy, x = m.normal(rows, n, dtype=dt), m.normal(rows, k, dtype=dt)
    to = torch.float32 if f32 else dt
    dw = m.place(E * n, k, to).view(E, n, k)
    hr.experts_product_grad(dy.to(DEV), x.to(DEV), dw, offsets=on_device(offsets))
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        d, v = dy[a:b].to(DEV).double(), x[a:b].to(DEV).double()
        ref, mag = (d.t() @ v).cpu(), (d.abs().t() @ v.abs()).cpu()
        within(dw[e], ref, sum_tol(to, ref, mag, b - a), f"dw of expert {e}")
    m.check_frames()
