"""GPU: every shape of tiles, in every type and layout, against 64 bits; the gradient's
stores past the caches; and large tiles in a captured graph."""
import pytest
import torch

from _gpu import needs_gpu
from _product_shapes import GRADIENTS, PRODUCTS
from _products import F8, sum_tol, wide_blocks, wide_rows
from _rows import TYPES, Maker
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"


def segments(rows, experts, seed):
    """Offsets of uneven segments, one without rows where there are several, and rows behind the last."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, rows - 1, (experts - 1,), generator=g)).values.tolist()
    if experts > 2:
        cuts[1] = cuts[0]
    return [0, *cuts, rows - (2 if experts > 2 else 0)]


def on_device(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device=DEV)


def inside(got, ref, mag, n, what, eight=False):
    """The bound of a sum of n products, on the GPU."""
    tol = sum_tol(got.dtype, ref, mag, n, eight=eight)
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), f"{what}: {int((~(off <= tol)).sum())} values off, worst {float((off / tol).max()):.3g} bounds"


def operands(m, kind, rows, k, shape):
    """(x, w, keywords, x and w as what they stand for)."""
    if kind != "e4m3":
        dt = TYPES[kind]
        x, w = m.normal(rows, k, dtype=dt).to(DEV), m.normal(*shape, dtype=dt).to(DEV)
        return x, w, {}, x.double(), w.double()
    x, w = (m.normal(*s, sigma=40.0).clamp(-448, 448).to(F8).to(DEV) for s in ((rows, k), shape))
    xs = torch.exp2(m.normal(rows, -(-k // 128)).clamp(-3, 3)).to(DEV)
    ws = torch.exp2(m.normal(shape[0], *(-(-v // 128) for v in shape[1:])).clamp(-3, 3) - 8).to(DEV)
    return x, w, dict(x_scales=xs, w_scales=ws), wide_rows(x, xs), wide_blocks(w, ws)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("along,across,experts,rows,k,n", PRODUCTS)
def test_product(kind, transposed, along, across, experts, rows, k, n):
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    m = Maker(rows + n)
    offsets = segments(rows, experts, n)
    x, w, scales, xw, ww = operands(m, kind, rows, k, (experts, *((k, n) if transposed else (n, k))))
    if along.startswith("Any"):                                  # at odd addresses too, rows apart
        buf = torch.full((rows * (k + 2) + 1,), 0x7F, dtype=torch.uint8, device=DEV).view(F8) if kind == "e4m3" else \
            torch.full((rows * (k + 2) + 1,), float("nan"), dtype=dt, device=DEV)
        apart = buf.as_strided((rows, k), (k + 2, 1), 1)
        apart.view(torch.uint8 if kind == "e4m3" else torch.int16).copy_(x.view(torch.uint8 if kind == "e4m3" else torch.int16))
        x = apart
    out = m.place(rows, n, dt, stride=n + 3, offset=1)
    hr.experts_product(x, w, out, offsets=on_device(offsets), transposed=transposed, **scales)
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        v = ww[e] if transposed else ww[e].t()
        inside(out[a:b], xw[a:b] @ v, xw[a:b].abs() @ v.abs(), k, f"expert {e}", eight=kind == "e4m3")
    assert (out[offsets[-1]:] == 7).all(), "wrote rows of no segment"
    m.check_frames()


def gradient(name, f32, experts, rows, n, k, offsets, seed):
    dt = TYPES[name]
    m = Maker(seed)
    dy, x = m.normal(rows, n, dtype=dt).to(DEV), m.normal(rows, k, dtype=dt).to(DEV)
    to = torch.float32 if f32 else dt
    buf = torch.full((2 + experts * (n * (k + 8) + 16),), 7.0, dtype=to, device=DEV)
    dw = buf.as_strided((experts, n, k), (n * (k + 8) + 16, k + 8, 1), 2)
    hr.experts_product_grad(dy, x, dw, offsets=on_device(offsets))
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        d, v = dy[a:b].double().t(), x[a:b].double()
        inside(dw[e], d @ v, d.abs() @ v.abs(), b - a, f"dw of expert {e}")
    dw.fill_(7.0)
    assert (buf == 7).all(), "wrote between the rows or the matrices"


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("shape,experts,rows,n,k", GRADIENTS)
def test_gradient(name, f32, shape, experts, rows, n, k):
    gradient(name, f32, experts, rows, n, k, segments(rows, experts, n), rows)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n", [840, 896, 1000])
def test_gradient_past_the_caches(name, f32, n):
    """dw of more than 256 MiB: several tiles a workgroup, with the last tiles' rows fewer than 128, 128 and more."""
    k, size = 3400, 4 if f32 else 2
    experts = -(-(1 << 28) // (n * k * size)) + 1
    assert experts * -(-n // 256) * -(-k // 256) > 3 * 256
    rows = 6000
    offsets = segments(rows, experts, n)
    offsets[5:9] = [offsets[4]] * 4                              # several of none in a row
    gradient(name, f32, experts, rows, n, k, offsets, n)


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_large_tiles_captured(kind):
    """Large tiles in a graph, replayed with fresh values and offsets, beside eager calls."""
    m, E, rows, k, n = Maker(6), 100, 20000, 528, 528
    dt = torch.float16
    x, w, scales, _, _ = operands(m, kind, rows, k, (E, n, k))
    dy = m.normal(rows, n, dtype=dt).to(DEV)
    xh = m.normal(rows, k, dtype=dt).to(DEV)
    at = on_device(segments(rows, E, 0))
    out, back, dw = torch.zeros(rows, n, dtype=dt, device=DEV), torch.zeros(rows, k, dtype=dt, device=DEV), \
        torch.empty(E, n, k, dtype=dt, device=DEV)

    def calls(out, back, dw, stream=None):
        hr.experts_product(x, w, out, offsets=at, stream=stream, **scales)
        hr.experts_product(x, w, back, offsets=at, transposed=True, stream=stream, **scales)
        hr.experts_product_grad(dy, xh, dw, offsets=at, stream=stream)

    calls(out, back, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(out, back, dw)
    side = torch.cuda.Stream()
    for i in range(4):
        raw = x.view(torch.uint8 if kind == "e4m3" else torch.int16)
        raw.copy_(raw.flip(0))
        dy.copy_(m.normal(rows, n, dtype=dt))
        xh.copy_(m.normal(rows, k, dtype=dt))
        at.copy_(torch.tensor(segments(rows, E, i), dtype=torch.int32))
        for t in (out, back, dw):
            t.zero_()
        mine = [torch.zeros_like(t) for t in (out, back, dw)]
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        calls(*mine, stream=side)
        torch.cuda.synchronize()
        for a, b in zip((out, back, dw), mine):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        o = at.tolist()
        for e in (0, 41, 99):
            d, v = dy[o[e]:o[e + 1]].double().t(), xh[o[e]:o[e + 1]].double()
            inside(dw[e], d @ v, d.abs() @ v.abs(), o[e + 1] - o[e], f"dw of expert {e}")
