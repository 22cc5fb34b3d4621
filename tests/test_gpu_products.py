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


def spread(rows, experts, seed):
    """Offsets of `rows` rows spread over the experts, unevenly."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, rows + 1, (experts - 1,), generator=g)).values.tolist()
    return [0, *cuts, rows]


# what every shape is chosen for: (experts, rows, k, n)
PICKS = [(1, 5, 264, 200), (8, 9, 136, 2008), (4, 40, 520, 3208), (1, 100, 328, 4104), (1, 250, 200, 2056),
         (16, 330, 72, 1288), (32, 1000, 136, 1288), (32, 2300, 200, 2056), (3, 700, 392, 520), (24, 5200, 136, 1032)]


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("experts,rows,k,n", PICKS)
def test_every_shape(kind, transposed, experts, rows, k, n):
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    m = Maker(rows + n)
    offsets = spread(rows, experts, n)
    if kind == "e4m3":
        k, n = k // 16 * 16, n // 16 * 16
        x, xs = eight(m, rows, k)
        ws = [eight(m, *((k, n) if transposed else (n, k)), blocks=True) for _ in range(experts)]
        w, wsc = torch.stack([a.view(torch.uint8) for a, _ in ws]).view(F8), torch.stack([b for _, b in ws]) * 2.0 ** -8
        scales = dict(x_scales=xs.to(DEV), w_scales=wsc.to(DEV))
        xw, ww = wide_rows(x, xs), wide_blocks(w, wsc)
    else:
        x, w = m.normal(rows, k, dtype=dt), m.normal(experts, *((k, n) if transposed else (n, k)), dtype=dt)
        scales, xw, ww = {}, x, w
    out = m.place(rows, n, dt)
    xd, wd, od = x.to(DEV), w.to(DEV), on_device(offsets)
    hr.experts_product(xd, wd, out, offsets=od, transposed=transposed, **scales)
    ref, mag = rows_ref(xw, ww, offsets, transposed)
    check_rows(m, out, ref, sum_tol(dt, ref, mag, k, eight=kind == "e4m3"), offsets, "out")
    again = torch.empty_like(out)
    hr.experts_product(xd, wd, again, offsets=od, transposed=transposed, **scales)
    assert torch.equal(again.view(torch.int16), out.reshape(rows, n).view(torch.int16)), "another result"


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("experts,rows,k,n", [(2, 3000, 200, 264), (12, 900, 648, 776), (60, 2000, 512, 512),
                                              (1, 5000, 136, 72)])
def test_every_shape_of_the_gradient(name, f32, experts, rows, k, n):
    dt = TYPES[name]
    m = Maker(rows + n)
    offsets = spread(rows, experts, n)
    dy, x = m.normal(rows, n, dtype=dt), m.normal(rows, k, dtype=dt)
    to = torch.float32 if f32 else dt
    dw = m.place(experts * n, k, to).view(experts, n, k)
    hr.experts_product_grad(dy.to(DEV), x.to(DEV), dw, offsets=on_device(offsets))
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        d, v = dy[a:b].to(DEV).double(), x[a:b].to(DEV).double()
        ref, mag = (d.t() @ v).cpu(), (d.abs().t() @ v.abs()).cpu()
        within(dw[e], ref, sum_tol(to, ref, mag, b - a), f"dw of expert {e}")
    m.check_frames()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("offset,extra", [(0, 8), (8, 16), (1, 3), (4, 12), (0, 1)])
@pytest.mark.parametrize("rows,k,n", [(40, 96, 136), (300, 136, 264)])
def test_strides_and_addresses(name, offset, extra, rows, k, n):
    """Rows apart, at any address of a value; matrices with room between them."""
    dt, E = TYPES[name], 3
    m = Maker(rows + extra)
    offsets = offsets_of([rows // 3, 0, rows - rows // 3 - 2])
    x, dy, w = m.normal(rows, k, dtype=dt), m.normal(rows, n, dtype=dt), m.normal(E, n, k, dtype=dt)
    xd = m.place(rows, k, dt, stride=k + extra, offset=offset, values=x)
    yd = m.place(rows, n, dt, stride=n + extra, offset=offset, values=dy)
    buf = torch.full((offset + E * (n + 2) * (k + extra) + 9,), 7.0, dtype=dt, device=DEV)
    strides = ((n + 2) * (k + extra), k + extra, 1)
    wd = buf.as_strided((E, n, k), strides, offset)
    wd.copy_(w)
    od = on_device(offsets)
    out, dx = m.place(rows, n, dt, stride=n + extra, offset=offset), m.place(rows, k, dt, stride=k + extra, offset=offset)
    hr.experts_product(xd, wd, out, offsets=od)
    hr.experts_product(yd, wd, dx, offsets=od, transposed=True)
    ref, mag = product_ref(x, w, offsets, False)
    check_rows(m, out, ref, sum_tol(dt, ref, mag, k), offsets, "out")
    ref, mag = product_ref(dy, w, offsets, True)
    check_rows(m, dx, ref, sum_tol(dt, ref, mag, n), offsets, "dx")
    hr.experts_product_grad(yd, xd, wd, offsets=od)                  # over the matrices themselves
    ref, mag = grad_ref(dy, x, offsets)
    within(wd.cpu(), ref, sum_tol(dt, ref, mag, rows), "dw")
    inside = torch.zeros(buf.numel(), dtype=torch.bool)
    inside.as_strided((E, n, k), strides, offset).fill_(True)
    assert (buf.cpu()[~inside] == 7).all(), "wrote between the matrices"


@pytest.mark.parametrize("offset,extra", [(0, 16), (16, 32), (1, 3), (4, 4)])
@pytest.mark.parametrize("rows,k,n", [(40, 160, 144), (300, 272, 272)])
def test_strides_and_addresses_8(offset, extra, rows, k, n):
    m = Maker(rows + extra)
    offsets = offsets_of([rows // 3, 0, rows - rows // 3 - 2])
    E = 3

    def place(codes, lead, stride):
        buf = torch.zeros(offset + lead * stride + 40, dtype=torch.uint8, device=DEV)
        view = buf.as_strided(codes.shape, (*((codes.shape[1] * stride,) if codes.dim() == 3 else ()), stride, 1), offset)
        view.copy_(codes.view(torch.uint8).to(DEV))
        return view.view(F8)

    x, xs = eight(m, rows, k)
    ws = [eight(m, n, k, blocks=True) for _ in range(E)]
    w, wsc = torch.stack([a.view(torch.uint8) for a, _ in ws]).view(F8), torch.stack([b for _, b in ws]) * 2.0 ** -8
    xd, wd = place(x, rows, k + extra), place(w, E * n, k + extra)
    xsd = m.place(rows, xs.shape[1], torch.float32, stride=xs.shape[1] + 3, offset=1, values=xs)
    out = m.place(rows, n, torch.bfloat16, stride=n + 7, offset=3)
    hr.experts_product(xd, wd, out, offsets=on_device(offsets), x_scales=xsd, w_scales=wsc.to(DEV))
    ref, mag = product_ref(wide_rows(x, xs), wide_blocks(w, wsc), offsets, False)
    check_rows(m, out, ref, sum_tol(torch.bfloat16, ref, mag, k, eight=True), offsets, "out")


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("rows,k,n", [(30, 144, 96), (200, 80, 272), (1200, 144, 1040)])
def test_what_is_not_finite_stays_in_its_row(kind, rows, k, n):
    """NaN and infinities beyond a segment, in one row, and beyond k."""
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    m = Maker(rows)
    offsets = offsets_of([rows // 2 - 1, 0, rows // 2 - 2])
    bad = [3, rows // 2]
    if kind == "e4m3":
        x, xs = eight(m, rows, k)
        ws = [eight(m, n, k, blocks=True) for _ in range(3)]
        w, wsc = torch.stack([a.view(torch.uint8) for a, _ in ws]).view(F8), torch.stack([b for _, b in ws])
        xs[bad[0], 0], xs[bad[1], -1] = float("nan"), float("inf")
        x.view(torch.uint8)[offsets[-1]:] = 0x7F                    # NaN
        scales = dict(x_scales=xs.to(DEV), w_scales=wsc.to(DEV))
        full = torch.full((rows, k + 16), 0x7F, dtype=torch.uint8)  # and NaN right behind every row
        full[:, :k] = x.view(torch.uint8)
        xd = full.to(DEV)[:, :k].view(F8)
        xw, ww = wide_rows(x, xs), wide_blocks(w, wsc)
    else:
        x, w = m.normal(rows, k, dtype=dt), m.normal(3, n, k, dtype=dt)
        x[bad[0], 5], x[bad[1], k - 1] = float("nan"), float("inf")
        x[offsets[-1]:] = float("nan")
        scales, xw, ww = {}, x, w
        full = torch.full((rows, k + 8), float("nan"), dtype=dt)
        full[:, :k] = x
        xd = full.to(DEV)[:, :k]
    out = m.place(rows, n, dt)
    hr.experts_product(xd, w.to(DEV), out, offsets=on_device(offsets), **scales)
    got = out.cpu().float()
    assert torch.isnan(got[bad[0]]).all() and not torch.isfinite(got[bad[1]]).any()
    xw = xw.clone()
    xw[bad] = 0
    ref, mag = product_ref(xw, ww, offsets, False)
    fine = torch.ones(rows, dtype=torch.bool)
    fine[bad] = False
    fine[offsets[-1]:] = False
    tol = sum_tol(dt, ref, mag, k, eight=kind == "e4m3")
    within(out.cpu()[fine], ref[fine], tol[fine], "other rows")
    if kind != "e4m3":
        dy = m.normal(rows, n, dtype=dt)
        dw = m.place(3 * n, k, dt).view(3, n, k)
        hr.experts_product_grad(dy.to(DEV), xd, dw, offsets=on_device(offsets))
        ref, mag = grad_ref(dy, x[:, :].masked_fill(~torch.isfinite(x), 0), offsets)
        tol = sum_tol(dt, ref, mag, rows)
        ref[0, :, 5] = float("nan")
        column = dw.cpu()[2, :, k - 1].float()
        assert not torch.isfinite(column).any()
        ref[2, :, k - 1], dwc = 0, dw.cpu().clone()
        dwc[2, :, k - 1] = 0
        within(dwc, ref, tol, "dw")


@pytest.mark.parametrize("offsets", [[0, 50, 20, 60], [-5, 10, 1 << 30, 30], [70, 60, 50, 40], [0, 64, 64, 65],
                                     [1 << 30, -1, 5, -7], [60, 64, 64, 64]])
@pytest.mark.parametrize("rows", [64, 640])
def test_any_offsets_stay_inside(offsets, rows):
    """Whatever the offsets hold, nothing outside the buffers is touched, and matrices without rows are zeros."""
    m, k, n = Maker(1), 72, 136
    dt = torch.float16
    x, w = m.normal(rows, k, dtype=dt).to(DEV), m.normal(3, n, k, dtype=dt).to(DEV)
    out, dw = m.place(rows, n, dt), m.place(3 * n, k, dt).view(3, n, k)
    at = on_device(offsets)
    hr.experts_product(x, w, out, offsets=at)
    hr.experts_product_grad(out, x, dw, offsets=at)
    act = m.place(rows, n // 2, dt)
    hr.experts_act(out, act, offsets=at)
    torch.cuda.synchronize()
    m.check_frames()
    for e in range(3):
        if min(max(offsets[e], 0), rows) >= min(offsets[e + 1], rows):
            assert (dw[e] == 0).all()


def test_no_rows():
    w = torch.ones(3, 16, 24, dtype=torch.float16, device=DEV)
    x, out = torch.empty(0, 24, dtype=torch.float16, device=DEV), torch.empty(0, 16, dtype=torch.float16, device=DEV)
    at = on_device([0, 0, 0, 0])
    hr.experts_product(x, w, out, offsets=at)
    hr.experts_product_grad(out, x, w, offsets=at)
    assert (w == 0).all()


def test_one_matrix_without_offsets():
    m = Maker(5)
    x, w = m.normal(70, 200, dtype=torch.float16), m.normal(136, 200, dtype=torch.float16)
    out = m.place(70, 136, torch.float16)
    hr.experts_product(x.to(DEV), w.to(DEV), out)
    ref, mag = product_ref(x, w[None], [0, 70], False)
    within(out.cpu(), ref, sum_tol(torch.float16, ref, mag, 200), "out")
    dw = m.place(136, 200, torch.float32)
    hr.experts_product_grad(out, x.to(DEV), dw)
    ref, mag = grad_ref(out.cpu(), x, [0, 70])
    within(dw.cpu(), ref[0], sum_tol(torch.float32, ref, mag, 70)[0], "dw")


def test_rows_past_two_to_the_32_bytes():
    """The last rows of buffers of more than 4 GiB, and matrices that lie as far apart."""
    k, n, rows = 64, 2056, (1 << 32) // 4096 + 700
    dt = torch.bfloat16
    out = torch.zeros(rows, n, dtype=dt, device=DEV)
    x = torch.zeros(rows, k, dtype=dt, device=DEV)
    m = Maker(9)
    last = m.normal(600, k, dtype=dt)
    x[rows - 600:] = last.to(DEV)
    w = m.normal(2, n, k, dtype=dt)
    far = torch.zeros((1 << 31) + n * k + 8, dtype=dt, device=DEV)
    wd = far.as_strided((2, n, k), (1 << 31, k, 1))
    wd.copy_(w)
    offsets = [rows - 600, rows - 300, rows]
    hr.experts_product(x, wd, out, offsets=on_device(offsets))
    ref, mag = product_ref(last, w, [0, 300, 600], False)
    within(out[rows - 600:].cpu(), ref, sum_tol(dt, ref, mag, k), "out")
    assert not out[:rows - 600].any()
    back = torch.zeros(rows, k, dtype=dt, device=DEV)
    hr.experts_product(out, wd, back, offsets=on_device(offsets), transposed=True)
    rounded = out[rows - 600:].cpu()
    ref, mag = product_ref(rounded, w, [0, 300, 600], True)
    within(back[rows - 600:].cpu(), ref, sum_tol(dt, ref, mag, n), "back")
    hr.experts_product_grad(out, x, wd, offsets=on_device(offsets))
    ref, mag = grad_ref(rounded, last, [0, 300, 600])
    within(wd.cpu(), ref, sum_tol(dt, ref, mag, 300), "dw")


def test_gradients_against_differences():
    """dx and dw of sum(dy * out), in float16 values that are exact in the sums."""
    m = Maker(3)
    offsets, k, n = [0, 5, 5, 12], 24, 16
    x, w, dy = (torch.randint(-4, 5, s, generator=m.g).to(torch.float16) for s in ((12, k), (3, n, k), (12, n)))

    def total(x, w):
        out = torch.empty(12, n, dtype=torch.float16, device=DEV)
        hr.experts_product(x.to(DEV), w.to(DEV), out, offsets=on_device(offsets))
        return float((out.cpu().double() * dy.double()).sum())

    dx, dw = torch.empty(12, k, dtype=torch.float16, device=DEV), torch.empty(3, n, k, dtype=torch.float32, device=DEV)
    hr.experts_product(dy.to(DEV), w.to(DEV), dx, offsets=on_device(offsets), transposed=True)
    hr.experts_product_grad(dy.to(DEV), x.to(DEV), dw, offsets=on_device(offsets))
    base = total(x, w)
    for r, c in ((0, 0), (4, 23), (5, 7), (11, 11)):
        y = x.clone()
        y[r, c] += 1
        assert total(y, w) - base == float(dx[r, c])
    for e, r, c in ((0, 0, 0), (1, 3, 3), (2, 15, 23)):
        v = w.clone()
        v[e, r, c] += 1
        assert total(x, v) - base == float(dw[e, r, c])


@pytest.mark.parametrize("k,n,E,rows", [(136, 264, 4, 700), (72, 1032, 12, 6000)])
def test_graphs_and_streams(k, n, E, rows):
    """Captured calls replayed with fresh inputs and offsets, beside eager ones on another stream."""
    m, dt = Maker(8), torch.bfloat16
    x, w, dy = (torch.empty(*s, dtype=dt, device=DEV) for s in ((rows, k), (E, n, k), (rows, n)))
    at = on_device([0] * (E + 1))
    out, dx, dw = torch.zeros(rows, n, dtype=dt, device=DEV), torch.zeros_like(x), torch.empty_like(w)

    def calls(out, dx, dw, stream=None):
        hr.experts_product(x, w, out, offsets=at, stream=stream)
        hr.experts_product(dy, w, dx, offsets=at, transposed=True, stream=stream)
        hr.experts_product_grad(dy, x, dw, offsets=at, stream=stream)

    calls(out, dx, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(out, dx, dw)
    side = torch.cuda.Stream()
    for i in range(4):
        x.copy_(m.normal(rows, k, dtype=dt))
        w.copy_(m.normal(E, n, k, dtype=dt))
        dy.copy_(m.normal(rows, n, dtype=dt))
        at.copy_(torch.tensor(spread(rows, E, i), dtype=torch.int32))
        torch.cuda.synchronize()
        mine = [torch.zeros_like(t) for t in (out, dx, dw)]
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        calls(*mine, stream=side)
        torch.cuda.synchronize()
        for a, b in zip((out, dx, dw), mine):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        ref, mag = product_ref(x.cpu(), w.cpu(), at.tolist(), False)
        within(out.cpu(), ref, sum_tol(dt, ref, mag, k), "out")


def test_most_rows():
    """As many rows as there may be, the last of them in a segment that begins just before."""
    rows, k, n = (1 << 31) - 4096, 8, 2
    x = torch.zeros(rows, k, dtype=torch.float16, device=DEV)
    at = [0, 1, 255, 256, 1 << 30, rows - 300, rows - 299, rows - 257, rows - 256, rows - 1]
    for i, r in enumerate(at):
        x[r] = i + 1
    w = torch.ones(2, n, k, dtype=torch.float16, device=DEV)
    w[1] = 2
    out = torch.full((rows, n), 7.0, dtype=torch.float16, device=DEV)
    hr.experts_product(x, w, out, offsets=on_device([0, rows - 299, rows]))
    for i, r in enumerate(at):
        assert (out[r] == (i + 1) * 8 * (2 if r >= rows - 299 else 1)).all()
        out[r] = 0
    for a in range(0, rows, 1 << 28):
        assert not out[a:a + (1 << 28)].any()


@pytest.mark.parametrize("kind", ["equal", "ties", "few", "any"])
def test_many_tiles_grad_in_any_order(kind):
    """Segments of equal and of unlike lengths, most of none, and offsets that go down again: five rounds of tiles."""
    m, dt, E, k, n, rows = Maker(len(kind)), torch.bfloat16, 300, 392, 512, 3000
    if kind == "any":
        offsets = torch.randint(-200, rows + 200, (E + 1,), generator=m.g).tolist()
    else:
        count = {"equal": torch.full((E,), 10), "ties": torch.arange(E) % 3 * 9, "few": torch.zeros(E, dtype=torch.int64)}[kind]
        if kind == "few":
            count[7], count[150], count[299] = 1000, 1500, 300
        offsets = offsets_of(count.tolist())
    dy, x = m.normal(rows, n, dtype=dt), m.normal(rows, k, dtype=dt)
    dw = m.place(E * n, k, dt).view(E, n, k)
    hr.experts_product_grad(dy.to(DEV), x.to(DEV), dw, offsets=on_device(offsets))
    dy, x = dy.to(DEV).float(), x.to(DEV).float()
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        a = min(max(a, 0), rows)
        b = max(min(b, rows), a)
        d, v = dy[a:b].double(), x[a:b].double()
        ref, mag = (d.t() @ v).cpu(), (d.abs().t() @ v.abs()).cpu()
        within(dw[e], ref, sum_tol(dt, ref, mag, b - a), f"dw of expert {e}")
    m.check_frames()


def test_gradient_of_a_very_large_matrix():
    """One row's outer product with more than 2^22 tiles and 2^36 values (137 GB)."""
    n = k = (1 << 18) + 1
    m = Maker(4)
    dy, x = m.normal(1, n, dtype=torch.bfloat16).to(DEV), m.normal(1, k, dtype=torch.bfloat16).to(DEV)
    torch.cuda.empty_cache()
    dw = torch.full((n, k), 7.0, dtype=torch.bfloat16, device=DEV)
    hr.experts_product_grad(dy, x, dw)
    for a in range(0, n, 1 << 13):
        d = dy[0, a:a + (1 << 13), None].float()
        # (one product, exact in binary32, rounded once)
        assert torch.equal(dw[a:a + (1 << 13)], (d * x.float()).to(torch.bfloat16)), f"rows {a} .."
    del dw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("k,n", [(136, 272), (135, 271), (1, 272), (136, 1), (1, 1)])
def test_one_row_with_a_large_distance(k, n, transposed):
    """Through the C entry: the distance of rows that are one row is not used."""
    m, dt, far = Maker(k + n), torch.float16, (1 << 32) + 8
    wr, wc = (k, n) if transposed else (n, k)
    x, w, dy = m.normal(1, k, dtype=dt), m.normal(1, wr, wc, dtype=dt), m.normal(1, n, dtype=dt)
    xd, wd, yd, out = x.to(DEV), w.to(DEV), dy.to(DEV), m.place(1, n, dt)
    a = hr.hr_experts_product_args()
    a.x, a.w, a.out, a.rows, a.n, a.k, a.experts = xd.data_ptr(), wd.data_ptr(), out.data_ptr(), 1, n, k, 1
    a.x_stride, a.out_stride, a.w_stride, a.transposed = far, far, far if wr == 1 else 0, int(transposed)
    stream = torch.cuda.current_stream().cuda_stream
    assert hr.hr_experts_product_f16(a, stream) == hr.HR_OK
    ref, mag = product_ref(x, w, [0, 1], transposed)
    within(out, ref, sum_tol(dt, ref, mag, k), "out")
    dw = m.place(n, k, dt)
    g = hr.hr_experts_product_grad_args()
    g.dy, g.x, g.dw, g.rows, g.n, g.k, g.experts = yd.data_ptr(), xd.data_ptr(), dw.data_ptr(), 1, n, k, 1
    g.dy_stride, g.x_stride, g.dw_stride = far, far, far if n == 1 else 0
    assert hr.hr_experts_product_grad_f16(g, stream) == hr.HR_OK
    ref, mag = grad_ref(dy, x, [0, 1])
    within(dw, ref[0], sum_tol(dt, ref, mag, 1)[0], "dw")
    m.check_frames()
