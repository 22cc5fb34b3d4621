"""hr_reduce_rmsnorm and hr_rmsnorm_grad on the GPU: the sum bit for bit
against the oracle's fold, the rest against the formulas in 64 bits, at row
lengths on both sides of every layout's limit, odd lengths, strides and
addresses, special values, and in place."""
import numpy as np
import pytest
import torch

from message_fp16_all_amd import hr
from _gpu import needs_gpu, specials_mix, specials_mix_bf16
from _rows import F32, TYPES, Maker, fold_ref, half_step, same, within

pytestmark = [pytest.mark.gpu, needs_gpu]

EPS = 1e-5
F8 = torch.float8_e4m3fn


def norm_ref(h, weight, eps=EPS):
    """(y, rstd) in 64 bits of 16-bit sums (CPU)."""
    x = h.double()
    rstd = 1.0 / torch.sqrt((x * x).mean(1) + eps)
    y = x * rstd[:, None]
    return (y if weight is None else y * weight.double().cpu()), rstd


def check_codes(codes, scales, y, group, what):
    """Scales against the largest magnitudes, codes against y / scale."""
    width = y.shape[1] if group == 0 else group
    c = codes.float().double().cpu()
    s = scales.double().cpu().reshape(y.shape[0], -1)
    parts = list(y.split(width, 1))
    assert s.shape[1] == len(parts), what
    for i, part in enumerate(parts):
        top = part.abs().amax(1)
        want = (top / 448).clamp_min(2.0 ** -126)
        within(s[:, i], want, want * F32, f"{what}: scale {i}")
        got = c[:, i * width:i * width + part.shape[1]] * s[:, i:i + 1]
        # half a step of e4m3: 2^-4 of the value, or half of its smallest, 2^-10
        tol = part.abs() * (2.0 ** -4 + F32) + s[:, i:i + 1] * 2.0 ** -10 * (1 + F32)
        within(got, torch.where(torch.isnan(s[:, i:i + 1]), torch.nan, part), tol, f"{what}: codes {i}")


def run_case(seed, dt, rows, hidden, G, residual=True, weight="same", group=None, out=True, stride=None, offset=0):
    m = Maker(seed)
    dtype = TYPES[dt]
    xs = [m.normal(rows, hidden, sigma=0.5, dtype=dtype) for _ in range(G)]
    r = m.normal(rows, hidden, dtype=dtype) if residual else None
    w = {"same": lambda: (m.normal(hidden, sigma=0.2) + 1).to(dtype), "f32": lambda: m.normal(hidden, sigma=0.2) + 1,
         "none": lambda: None}[weight]()
    dx = [m.place(rows, hidden, dtype, stride, offset, x) for x in xs]
    dr = m.place(rows, hidden, dtype, stride, offset + 1, r) if residual else None
    dw = m.place(1, hidden, w.dtype, None, offset, w[None])[0] if w is not None else None
    h = m.place(rows, hidden, dtype, stride, offset)
    y = m.place(rows, hidden, dtype, stride, offset + 3) if out else None
    rstd = torch.full((rows,), 9.0, device="cuda:0")
    codes = scales = None
    if group is not None:
        codes = m.place(rows, hidden, F8, stride, offset)
        n = -(-hidden // group) if group else 1
        scales = m.place(rows, n, torch.float32, n + 3 if stride else None, 1)
    print(f"norm {dt} {rows}x{hidden} G={G} residual={residual} weight={weight} group={group} stride={stride} "
          f"offset={offset}", flush=True)
    hr.reduce_rmsnorm(dx, y, residual=dr, residual_out=h, weight=dw, eps=EPS, out8=codes, scales=scales,
                      group=group or 0, rstd=rstd)
    torch.cuda.synchronize()
    href = fold_ref(xs + ([r] if residual else []))
    same(h, href, "h")
    yref, rref = norm_ref(href, w)
    within(rstd, rref, rref * F32, "rstd")
    if out:
        within(y, yref, half_step(dtype, yref) * (1 + F32) + yref.abs() * F32, "y")
    if group is not None:
        check_codes(codes, scales, yref, group, "e4m3")
    m.check_frames()


# both sides of every layout's limit: 16, 32 and 64 lanes per row, then a
# workgroup with one, two and four units per thread
WIDTHS = [1, 7, 8, 9, 64, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 2048, 4096, 4097, 5120, 6144, 8192, 16384,
          16385, 20001, 32767, 32768]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_widths(dt, hidden):
    run_case(hidden, dt, 5, hidden, 3, group=128)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", list(range(1, 17)))
def test_group_sizes(dt, G):
    for hidden in (128, 1024, 6144, 17000):
        run_case(100 + G, dt, 3, hidden, G, residual=G % 2 == 0, weight="f32", group=0)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 63, 64, 1000, 5003])
def test_rows(rows):
    run_case(rows, "bf16", rows, 128, 2, weight="none", group=32)
    run_case(rows, "f16", rows, 320, 1, residual=False, group=64)
    if rows <= 1000:
        run_case(rows, "bf16", rows, 5120, 2, group=0)


# both sides of 512 workgroups of 16, 8 and 4 rows and of one: how many operands
# a thread loads at once
@pytest.mark.parametrize("rows,hidden", [(8192, 72), (8193, 72), (4096, 200), (4097, 200), (2048, 511), (2049, 511),
                                         (512, 1032), (513, 1032)])
@pytest.mark.parametrize("G", [4, 10, 16])
def test_few_and_many_workgroups(rows, hidden, G):
    run_case(rows, "bf16", rows, hidden, G, group=64)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden,stride,offset", [(128, 130, 1), (500, 777, 3), (4096, 4099, 1), (5121, 5121, 5),
                                                  (9000, 9008, 7), (32768, 40001, 1)])
def test_strides_and_odd_addresses(dt, hidden, stride, offset):
    for group in (0, 128):
        run_case(hidden, dt, 7, hidden, 2, weight="f32", group=group, stride=stride, offset=offset)


def test_codes_alone():
    run_case(1, "bf16", 33, 6144, 8, group=128, out=False)
    run_case(2, "f16", 33, 200, 1, group=0, out=False)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_special_values(dt):
    """Infinities, NaN, subnormals and zeros: rows of each, and all together."""
    dtype = TYPES[dt]
    n = 2048
    make = specials_mix_bf16 if dt == "bf16" else specials_mix
    rows = [torch.from_numpy(make(n, s).view(np.int16).copy()).view(dtype) for s in (1, 2)]
    tiny = torch.finfo(dtype).tiny
    z = torch.zeros(n, dtype=dtype)
    one = {"inf": float("inf"), "-inf": float("-inf"), "nan": float("nan")}
    x = [rows[0], z, z + tiny / 4, -z]
    for v in one.values():
        r = torch.linspace(-3, 3, n).to(dtype)
        r[777] = v
        x.append(r)
    x = torch.stack(x)
    res = torch.zeros_like(x)
    res[0] = rows[1]
    dev = "cuda:0"
    h, y, codes = (torch.empty(x.shape, dtype=t, device=dev) for t in (dtype, dtype, F8))
    scales, rstd = torch.empty(len(x), 16, device=dev), torch.empty(len(x), device=dev)
    hr.reduce_rmsnorm([x.to(dev)], y, residual=res.to(dev), residual_out=h, eps=EPS, out8=codes, scales=scales,
                      group=128, rstd=rstd)
    torch.cuda.synchronize()
    href = fold_ref([x, res])
    same(h, href, "h")
    # squares are summed in 32 bits: the reference says so where they pass its range
    f = href.float()
    rref = (1.0 / torch.sqrt((f * f).mean(1) + EPS)).double()
    yref = href.double() * rref[:, None]
    ok = torch.isfinite(href).all(1)
    within(rstd, rref, rref.abs() * 2 * F32, "rstd")
    within(y[ok.to(dev)], yref[ok], half_step(dtype, yref[ok]) + yref[ok].abs() * 3 * F32, "y")
    assert torch.equal(torch.isnan(y).cpu(), torch.isnan(yref)), "NaN where the formula gives NaN"
    # the zero rows: codes 0 and the smallest scale
    assert (codes[1].float() == 0).all() and (scales[1] == 2.0 ** -126).all()
    # the groups with a NaN have a NaN scale and NaN codes; a row with an infinity is zero elsewhere
    for i, v in enumerate(one.values()):
        g = 777 // 128
        assert torch.isnan(scales[4 + i, g]) and torch.isnan(codes[4 + i, 777].float())
        if v == v:
            assert (codes[4 + i, :128].float() == 0).all()
        else:
            assert torch.isnan(codes[4 + i].float()).all()


@pytest.mark.parametrize("hidden", [128, 4096, 9001, 20000])
def test_in_place(hidden):
    """residual_out over the residual, out over a contribution; and out over
    the residual beside residual_out over a contribution."""
    m = Maker(hidden)
    rows, dtype = 9, torch.bfloat16
    xs = [m.normal(rows, hidden, dtype=dtype) for _ in range(3)]
    r = m.normal(rows, hidden, dtype=dtype)
    href = fold_ref(xs + [r])
    yref, _ = norm_ref(href, None)
    for swap in (False, True):
        dx, dr = [x.cuda() for x in xs], r.cuda()
        h, y = (dx[1], dr) if swap else (dr, dx[1])
        hr.reduce_rmsnorm(dx, y, residual=dr, residual_out=h, eps=EPS)
        torch.cuda.synchronize()
        same(h, href, "h")
        within(y, yref, half_step(dtype, yref) + yref.abs() * F32, "y")


def test_same_bits_as_reduce():
    m = Maker(5)
    xs = [m.normal(64, 6144, dtype=torch.float16).cuda() for _ in range(9)]
    out, h = torch.empty_like(xs[0]), torch.empty_like(xs[0])
    hr.reduce(xs, out)
    hr.reduce_rmsnorm(xs[:8], residual=xs[8], residual_out=h)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), h.view(torch.int16))


def test_no_rows_and_other_shapes():
    x = torch.zeros(0, 64, dtype=torch.float16, device="cuda:0")
    hr.reduce_rmsnorm([x], torch.empty_like(x))
    x = torch.randn(2, 3, 40, 128, device="cuda:0").half()      # heads, contiguous
    y = torch.empty_like(x)
    hr.reduce_rmsnorm([x], y, eps=EPS)
    ref, _ = norm_ref(x.cpu().reshape(-1, 128), None)
    within(y.reshape(-1, 128), ref, half_step(torch.float16, ref) + ref.abs() * F32, "heads")
    v = torch.randn(4096, device="cuda:0").half()               # one row
    y = torch.empty_like(v)
    hr.reduce_rmsnorm([v], y, eps=EPS)
    ref, _ = norm_ref(v.cpu()[None], None)
    within(y[None], ref, half_step(torch.float16, ref) + ref.abs() * F32, "one row")


def test_far_rows():
    """Offsets past 2^32 bytes (and past 2^31 values) of a strided buffer."""
    hidden, stride, rows = 256, (1 << 31) + 24, 2
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    buf = torch.empty(stride + hidden, dtype=torch.float16, device="cuda:0")
    view = buf.as_strided((rows, hidden), (stride, 1))
    x = torch.randn(rows, hidden).half()
    view.copy_(x)
    y = torch.empty(rows, hidden, dtype=torch.float16, device="cuda:0")
    hr.reduce_rmsnorm([view], y, residual_out=view, eps=EPS)
    ref, _ = norm_ref(x, None)
    within(y, ref, half_step(torch.float16, ref) + ref.abs() * F32, "y")
    same(view, x, "h")


# ------------------------------------------------------------------ gradient

def grad_ref(dy, h, rstd, w, dres):
    """dx, dweight in 64 bits, and the magnitudes that went into them."""
    dy, h, r = dy.double(), h.double(), rstd.double().cpu()[:, None]
    g = dy * (w.double() if w is not None else 1.0)
    u = h * r
    mean = (g * u).mean(1, keepdim=True)
    dx = r * (g - u * mean)
    size = r * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    if dres is not None:
        dx, size = dx + dres.double(), size + dres.double().abs()
    return dx, size, (dy * u).sum(0), (dy * u).abs().sum(0)


def run_grad(seed, dt, rows, hidden, weight="same", dres=True, stride=None, offset=0, in_place=None, workspace=True):
    m = Maker(seed)
    dtype = TYPES[dt]
    dy, h = m.normal(rows, hidden, sigma=0.3, dtype=dtype), m.normal(rows, hidden, sigma=2.0, dtype=dtype)
    r = m.normal(rows, hidden, sigma=0.3, dtype=dtype) if dres else None
    w = {"same": lambda: (m.normal(hidden, sigma=0.2) + 1).to(dtype), "f32": lambda: m.normal(hidden, sigma=0.2) + 1,
         "none": lambda: None}[weight]()
    rstd = (1.0 / torch.sqrt(h.float().square().mean(1) + EPS)).cuda()
    d = {"dy": m.place(rows, hidden, dtype, stride, offset, dy), "h": m.place(rows, hidden, dtype, stride, offset + 1, h),
         "dres": m.place(rows, hidden, dtype, stride, offset, r) if dres else None}
    dx = d[in_place] if in_place else m.place(rows, hidden, dtype, stride, offset + 3)
    dw = m.place(1, hidden, torch.float32, None, 1)[0]
    ws = None
    if workspace:
        # dirty, so that nothing is taken for granted
        ws = torch.full((hr.hr_rmsnorm_grad_workspace(rows, hidden) + 64,), 255, dtype=torch.uint8, device="cuda:0")
    print(f"norm grad {dt} {rows}x{hidden} weight={weight} dres={dres} stride={stride} in_place={in_place}", flush=True)
    hr.rmsnorm_grad(d["dy"], d["h"], rstd, dx, weight=w.cuda() if w is not None else None, dresidual=d["dres"],
                    dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    ref, size, wref, wsize = grad_ref(dy, h, rstd, w, r)
    within(dx, ref, half_step(dtype, ref) * (1 + F32) + size * 2 * F32, "dx")
    # a column's sum: at most rows additions in sequence and 16 more
    within(dw, wref, wsize * (rows + 32) * 2.0 ** -24, "dweight")
    m.check_frames()
    return dx.clone(), dw.clone()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_grad_widths(dt, hidden):
    run_grad(hidden, dt, 5, hidden)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 511, 512, 513, 8193, 20000])
def test_grad_rows(rows):
    run_grad(rows, "bf16", rows, 128, weight="f32", dres=False)
    run_grad(rows, "f16", rows, 257, weight="none")
    if rows < 8000:
        run_grad(rows, "f16", rows, 4096)
        run_grad(rows, "bf16", rows, 8200, weight="f32", workspace=False)


# short and long rows, with one, two and more workgroups on a compute unit
@pytest.mark.parametrize("rows,hidden", [(513, 2048), (514, 2048), (700, 2049), (1024, 2048), (1031, 2047), (2100, 1327),
                                         (4100, 300), (8200, 200), (16400, 64), (40000, 65)])
def test_grad_workgroups(rows, hidden):
    run_grad(rows, "bf16", rows, hidden, weight="f32")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden,stride,offset", [(128, 130, 1), (500, 777, 3), (5121, 5121, 5), (32767, 40001, 1)])
def test_grad_strides(dt, hidden, stride, offset):
    run_grad(hidden, dt, 19, hidden, weight="f32", stride=stride, offset=offset)


@pytest.mark.parametrize("what", ["dy", "h", "dres"])
def test_grad_in_place(what):
    for hidden in (128, 4096, 20000):
        run_grad(3, "f16", 700, hidden, in_place=what)
        run_grad(4, "bf16", 100, hidden + 1, in_place=what)
        run_grad(5, "f16", 100, hidden, in_place=what, workspace=False)


def test_grad_of_few_rows_takes_no_workspace():
    """Up to HR_RMSNORM_GRAD_FEW_ROWS rows dweight is summed beside dx, and a row more is not."""
    limit = hr.HR_RMSNORM_GRAD_FEW_ROWS
    for rows in (1, 15, 17, limit - 1, limit):
        for hidden in (7, 128, 129, 1000, 4100):
            run_grad(rows, "bf16", rows, hidden, weight="f32", workspace=False)
    h = torch.ones(limit + 1, 1024, dtype=torch.float16, device="cuda:0")
    args = [t.data_ptr() for t in (h, h)]
    a = hr.hr_rmsnorm_grad_args()
    dx, dw, rstd = torch.empty_like(h), torch.empty(1024, device="cuda:0"), torch.ones(limit + 1, device="cuda:0")
    a.dy, a.h, a.rstd, a.dx, a.dweight = *args, rstd.data_ptr(), dx.data_ptr(), dw.data_ptr()
    a.hidden = 1024
    for rows, into, status in ((limit, dx, hr.HR_OK), (limit + 1, dx, hr.HR_ERR_INVALID_ARG),
                               (limit, h, hr.HR_ERR_INVALID_ARG)):
        a.rows, a.dx = rows, into.data_ptr()
        assert hr.hr_rmsnorm_grad_f16(a, torch.cuda.current_stream().cuda_stream) == status
    torch.cuda.synchronize()
    assert (dw == limit).all()


def test_grad_is_the_same_every_time():
    a = run_grad(9, "bf16", 5003, 1024)
    b = run_grad(9, "bf16", 5003, 1024)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_grad_without_rows_or_weight_gradient():
    dw = torch.full((96,), 5.0, device="cuda:0")
    e = torch.zeros(0, 96, dtype=torch.float16, device="cuda:0")
    hr.rmsnorm_grad(e, e, torch.zeros(0, device="cuda:0"), torch.empty_like(e), dweight=dw)
    assert (dw == 0).all()
    m = Maker(4)
    h, dy = m.normal(40, 96, dtype=torch.float16), m.normal(40, 96, dtype=torch.float16)
    rstd = (1.0 / torch.sqrt(h.float().square().mean(1) + EPS)).cuda()
    dx = torch.empty(40, 96, dtype=torch.float16, device="cuda:0")
    hr.rmsnorm_grad(dy.cuda(), h.cuda(), rstd, dx)
    ref, size, _, _ = grad_ref(dy, h, rstd, None, None)
    within(dx, ref, half_step(torch.float16, ref) + size * 2 * F32, "dx")


def test_grad_against_differences():
    """dx and dweight against central differences of the forward formula in 64
    bits.  A difference's own error is step^2 / 6 times the third derivative,
    far below the 16-bit rounding at step 1e-4 for values of order one."""
    m = Maker(12)
    rows, hidden, step = 2, 24, 1e-4
    h, dy = m.normal(rows, hidden, dtype=torch.float16), m.normal(rows, hidden, dtype=torch.float16)
    w = m.normal(hidden) + 1
    x = h.double()

    def loss(x, w):
        return (x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w * dy.double()).sum()

    ref = torch.zeros(rows, hidden, dtype=torch.float64)
    wref = torch.zeros(hidden, dtype=torch.float64)
    for i in range(rows):
        for j in range(hidden):
            e = torch.zeros_like(x)
            e[i, j] = step
            ref[i, j] = (loss(x + e, w.double()) - loss(x - e, w.double())) / (2 * step)
    for j in range(hidden):
        e = torch.zeros(hidden, dtype=torch.float64)
        e[j] = step
        wref[j] = (loss(x, w.double() + e) - loss(x, w.double() - e)) / (2 * step)
    out, hh, rstd = (torch.empty(rows, hidden, dtype=torch.float16, device="cuda:0") for _ in range(2)), None, None
    y, hh = out
    rstd = torch.empty(rows, device="cuda:0")
    hr.reduce_rmsnorm([h.cuda()], y, residual_out=hh, weight=w.cuda(), eps=EPS, rstd=rstd)
    dx, dw = torch.empty_like(hh), torch.empty(hidden, device="cuda:0")
    hr.rmsnorm_grad(dy.cuda(), hh, rstd, dx, weight=w.cuda(), dweight=dw)
    _, size, _, wsize = grad_ref(dy, h, rstd, w, None)
    within(dx, ref, half_step(torch.float16, ref) + size * 2 * F32 + 1e-6, "dx")
    within(dw, wref, wsize * 64 * 2.0 ** -24 + 1e-6, "dweight")


# ------------------------------------------------------------ streams, graphs

def test_another_stream_and_a_graph():
    m = Maker(21)
    rows, hidden = 300, 4096
    xs = [m.normal(rows, hidden, dtype=torch.float16).cuda() for _ in range(2)]
    w = (m.normal(hidden, sigma=0.1) + 1).cuda()
    h, y, dx = (torch.empty_like(xs[0]) for _ in range(3))
    rstd, dw = torch.empty(rows, device="cuda:0"), torch.empty(hidden, device="cuda:0")
    ws = torch.empty(hr.hr_rmsnorm_grad_workspace(rows, hidden), dtype=torch.uint8, device="cuda:0")

    def step(stream=None, workspace=None):
        hr.reduce_rmsnorm(xs, y, residual_out=h, weight=w, rstd=rstd, stream=stream)
        hr.rmsnorm_grad(y, h, rstd, dx, weight=w, dweight=dw, workspace=workspace, stream=stream)

    def eager():
        step()
        torch.cuda.synchronize()
        return [t.clone() for t in (h, y, dx, rstd, dw)]

    first = eager()
    s = torch.cuda.Stream()
    for t in (h, y, dx, rstd, dw):
        t.zero_()
    torch.cuda.synchronize()
    step(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (h, y, dx, rstd, dw)))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(workspace=ws)
    for k in range(4):
        for x in xs:
            x.copy_(m.normal(rows, hidden, dtype=torch.float16))
        want = eager()
        for t in (h, y, dx, rstd, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (h, y, dx, rstd, dw))), f"replay {k}"


# ------------------------------------------------------------------ refusals

def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda:0")
    y = torch.empty_like(x)
    for bad, err in [(lambda: hr.reduce_rmsnorm([x.float()], y), TypeError),
                     (lambda: hr.reduce_rmsnorm([x, x.bfloat16()], y), TypeError),
                     (lambda: hr.reduce_rmsnorm([x], y.bfloat16()), TypeError),
                     (lambda: hr.reduce_rmsnorm([x], y.cpu()), TypeError),
                     (lambda: hr.reduce_rmsnorm([x], y[:3]), ValueError),
                     (lambda: hr.reduce_rmsnorm([x], y.t()), ValueError),
                     (lambda: hr.reduce_rmsnorm([x[:1].expand(4, 64)], y), ValueError),
                     (lambda: hr.reduce_rmsnorm([x, x[:, :64].clone().repeat(1, 2)[:, :64]], y), ValueError),
                     (lambda: hr.reduce_rmsnorm([x] * 17, y), ValueError),
                     (lambda: hr.reduce_rmsnorm([x], y, weight=torch.ones(63, device="cuda:0")), ValueError),
                     (lambda: hr.reduce_rmsnorm([x], y, weight=torch.ones(64, device="cuda:0").double()), TypeError),
                     (lambda: hr.reduce_rmsnorm([x], y, rstd=torch.ones(3, device="cuda:0")), ValueError),
                     (lambda: hr.reduce_rmsnorm([x], y, out8=torch.empty(4, 64, dtype=F8, device="cuda:0")),
                      hr.HrError),
                     (lambda: hr.reduce_rmsnorm([x], y, out8=y, scales=torch.ones(4, device="cuda:0")), TypeError),
                     (lambda: hr.reduce_rmsnorm([x], y, eps=-1.0), hr.HrError),
                     (lambda: hr.reduce_rmsnorm([x]), hr.HrError),
                     (lambda: hr.rmsnorm_grad(y, x, torch.ones(4, device="cuda:0"), y.bfloat16()), TypeError),
                     (lambda: hr.rmsnorm_grad(y, x, torch.ones(5, device="cuda:0"), y), ValueError),
                     (lambda: hr.rmsnorm_grad(y, x, torch.ones(4, device="cuda:0"), y,
                                              dweight=torch.ones(64, device="cuda:0").half()), TypeError)]:
        with pytest.raises(err):
            bad()
    hr.reduce_rmsnorm([x + 1], y, eps=0.0)
    torch.cuda.synchronize()
    assert (y == 1).all()


# ------------------------------------------------------------------ 8 bits

# one row to a wave's lanes and to a workgroup, whole units and odd lengths, and
# (the last) rows that pass the caches by
@pytest.mark.parametrize("rows,hidden,group", [(33, 128, 32), (33, 129, 0), (9, 1000, 64), (9, 1001, 128),
                                               (7, 5120, 128), (7, 5121, 0), (3, 20000, 0), (3, 20001, 32),
                                               (8200, 4096, 128)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_codes_at_ties(dt, rows, hidden, group):
    """Values whose ratio to the largest lies half way between two codes: the
    codes are e4m3 of the binary32 quotient y / scale, to the bit.  (y is the
    two binary32 products that the formula names, so it can be had from rstd.)"""
    g = torch.Generator().manual_seed(hidden)

    def rand(low, high):
        return torch.randint(low, high, (rows, hidden), generator=g)

    # five significant bits: every odd one is a tie of codes' four
    x = (rand(16, 32) * 2.0 ** rand(-4, 5)).clamp(max=448.0) * (2 * rand(0, 2) - 1)
    width = group or hidden
    x[:, ::width] = 448.0
    x = x.to(TYPES[dt])
    w = torch.tensor([0.75, 1.0, 1.3])[torch.arange(-(-hidden // width)) % 3].repeat_interleave(width)[:hidden]
    codes = torch.empty(rows, hidden, dtype=F8, device="cuda:0")
    n = -(-hidden // width)
    scales, rstd = torch.empty(rows, n, device="cuda:0"), torch.empty(rows, device="cuda:0")
    print(f"ties {dt} {rows}x{hidden} group={group}", flush=True)
    hr.reduce_rmsnorm([x.cuda()], torch.empty_like(x, device="cuda:0"), weight=w.cuda(), eps=EPS, out8=codes,
                      scales=scales, group=group, rstd=rstd)
    torch.cuda.synchronize()
    y = x.float() * rstd.cpu()[:, None] * w
    top = torch.stack([part.abs().amax(1) for part in y.split(width, 1)], 1)
    assert torch.equal(scales.cpu(), top / 448)
    want = (y / scales.cpu().repeat_interleave(width, 1)[:, :hidden]).to(F8)
    bad = codes.cpu().view(torch.uint8) != want.view(torch.uint8)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes are not the quotient's"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_codes_over_the_range_of_scales(dt):
    """The same from the smallest scale to an infinite one, zeros of both signs
    among the values."""
    exps = [-148, -140, -130, -126, -118, -110, -100, -95, -92, -91, -90, -89, -60, 0, 60, 100, 115, 119, 121, 124, 126,
            127]
    g = torch.Generator().manual_seed(5)
    rows, group = 64, 32
    hidden = group * len(exps)
    x = torch.randint(16, 32, (rows, hidden), generator=g) * 2.0 ** torch.randint(-14, 5, (rows, hidden), generator=g)
    x = x.clamp(max=448.0) * (2 * torch.randint(0, 2, (rows, hidden), generator=g) - 1)
    x[:, ::group], x[:, 1::group], x[:, 2::group] = 448.0, 0.0, -0.0
    x = x.to(TYPES[dt])
    w = torch.tensor([2.0 ** e for e in exps]).repeat_interleave(group)
    codes, scales = torch.empty(rows, hidden, dtype=F8, device="cuda:0"), torch.empty(rows, len(exps), device="cuda:0")
    rstd = torch.empty(rows, device="cuda:0")
    hr.reduce_rmsnorm([x.cuda()], weight=w.cuda(), eps=EPS, out8=codes, scales=scales, group=group, rstd=rstd)
    torch.cuda.synchronize()
    y = x.float() * rstd.cpu()[:, None] * w
    s = (y.abs().view(rows, -1, group).amax(2) / 448).clamp_min(2.0 ** -126)
    assert torch.isinf(s).any() and (s == 2.0 ** -126).any()
    assert torch.equal(scales.cpu(), s)
    want, got = (y.view(rows, -1, group) / s[:, :, None]).view(rows, hidden).to(F8), codes.cpu()
    nan = torch.isnan(want.float())
    assert torch.equal(torch.isnan(got.float()), nan) and nan.any()
    bad = (got.view(torch.uint8) != want.view(torch.uint8)) & ~nan
    assert not bad.any(), f"{int(bad.sum())} codes, the first of w = 2^{exps[int(bad.nonzero()[0, 1]) // group]}"


# --------------------------------------------------- calls that pass the caches by

STREAMED = 1 << 27               # bytes moved from which they do
STREAMED_WIDTHS = [121, 128, 250, 256, 505, 512, 4001, 4096, 8190, 8192, 20000, 20001]


def rows_buffer(g, rows, hidden, dtype, pad, offset, sigma=1.0):
    """Random values all over a buffer, and the rows in it: `pad` values between
    two of them, the first at `offset`."""
    buf = torch.empty(offset + rows * (hidden + pad) + 8, dtype=dtype, device="cuda:0").normal_(0, sigma, generator=g)
    return buf, lambda b, a=0, n=rows: b.as_strided((n, hidden), (hidden + pad, 1), offset + a * (hidden + pad))


def parts_of(rows):
    """Four parts, each a call below the limit."""
    cuts = [rows * i // 4 for i in range(5)]
    return [(a, b - a) for a, b in zip(cuts, cuts[1:])]


def equal(a, b, what):
    same_bits = a.view(torch.uint8) == b.view(torch.uint8)
    assert same_bits.all(), f"{what}: {int((~same_bits).sum())} bytes differ"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden", STREAMED_WIDTHS)
def test_streamed_norm(dt, hidden):
    """One large call gives the bits of its parts, and leaves what lies around
    its rows alone: packed and strided, apart and in place."""
    dtype, g = TYPES[dt], torch.Generator(device="cuda:0").manual_seed(hidden)
    rows = STREAMED // (hidden * 2 * 5) + 3          # 5 arrays of rows
    w = torch.empty(hidden, device="cuda:0").normal_(1, 0.2, generator=g)
    for pad, offset, group in ((0, 0, 128), (5, 1, 0), (8, 8, 64)):
        print(f"streamed norm {dt} {rows}x{hidden} pad={pad} group={group}", flush=True)
        (x, view), (r, _) = (rows_buffer(g, rows, hidden, dtype, pad, offset) for _ in range(2))
        n = -(-hidden // group) if group else 1
        got = []
        for parts in ([(0, rows)], parts_of(rows)):
            h, y = (torch.full_like(x, 7) for _ in range(2))
            codes = torch.full(x.shape, 7, dtype=torch.uint8, device="cuda:0").view(F8)
            scales, rstd = torch.full((rows, n), 7.0, device="cuda:0"), torch.full((rows,), 7.0, device="cuda:0")
            x2, r2 = x.clone(), r.clone()
            for a, m in parts:
                hr.reduce_rmsnorm([view(x, a, m)], view(y, a, m), residual=view(r, a, m), residual_out=view(h, a, m),
                                  weight=w, eps=EPS, out8=view(codes, a, m), scales=scales[a:a + m], group=group,
                                  rstd=rstd[a:a + m])
                hr.reduce_rmsnorm([view(x2, a, m)], view(x2, a, m), residual=view(r2, a, m), residual_out=view(r2, a, m),
                                  weight=w, eps=EPS, out8=view(codes, a, m), scales=scales[a:a + m], group=group)
            torch.cuda.synchronize()
            equal(view(y).contiguous(), view(x2).contiguous(), "out in place")
            equal(view(h).contiguous(), view(r2).contiguous(), "h in place")
            got.append((h, y, codes, scales, rstd, x2, r2))
        for name, a, b in zip(("h", "y", "codes", "scales", "rstd", "out in place", "h in place"), *got):
            equal(a, b, name)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden", STREAMED_WIDTHS)
def test_streamed_grad(dt, hidden):
    """dx of one large call has the bits of its parts, in place too; dweight
    against the formula in 64 bits."""
    dtype, g = TYPES[dt], torch.Generator(device="cuda:0").manual_seed(hidden)
    rows = STREAMED // (hidden * 2 * 4) + 3          # dy, h, dresidual and dx
    w = torch.empty(hidden, device="cuda:0").normal_(1, 0.2, generator=g)
    for pad, offset in ((0, 0), (5, 1)):
        print(f"streamed norm grad {dt} {rows}x{hidden} pad={pad}", flush=True)
        made = [rows_buffer(g, rows, hidden, dtype, pad, offset) for _ in range(3)]
        view = made[0][1]
        dy, h, r = (b for b, _ in made)
        rstd = 1.0 / torch.sqrt(view(h).float().square().mean(1) + EPS)
        first = torch.full_like(dy, 7)
        for a, m in parts_of(rows):
            hr.rmsnorm_grad(view(dy, a, m), view(h, a, m), rstd[a:a + m], view(first, a, m), weight=w,
                            dresidual=view(r, a, m))
        prod = view(dy).double() * (view(h).double() * rstd.double()[:, None])
        ref, size = prod.sum(0).cpu(), prod.abs().sum(0).cpu()
        del prod
        for into in (None, 0, 1, 2):
            d = [b.clone() for b in (dy, h, r)]
            out = torch.full_like(dy, 7) if into is None else d[into]
            dw = torch.full((hidden,), 7.0, device="cuda:0")
            hr.rmsnorm_grad(view(d[0]), view(d[1]), rstd, view(out), weight=w, dresidual=view(d[2]), dweight=dw)
            torch.cuda.synchronize()
            want = first if into is None else (dy, h, r)[into].clone()
            view(want).copy_(view(first))
            equal(out, want, f"dx into {into}")
            within(dw, ref, size * (rows + 32) * 2.0 ** -24, "dweight")
