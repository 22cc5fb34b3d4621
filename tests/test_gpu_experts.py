"""hr_experts_sort, _gather, _combine and _combine_grad on the GPU: the sort and
the copies exactly, the sums against the formulas in 64 bits; one workgroup's
sort and many workgroups', padding, dropped and foreign picks, odd row lengths,
strides and addresses, rows past 2^32 bytes."""
import numpy as np
import pytest
import torch

from message_fp16_all_amd import hr
from _gpu import needs_gpu
from _rows import TYPES, Maker, half_step, within

pytestmark = [pytest.mark.gpu, needs_gpu]

DEV = "cuda:0"
F32 = 2.0 ** -24


def sort_reference(ids, first, experts, pad, rows):
    """(offsets, order, pos) of the definition, in numpy."""
    ids = ids.reshape(-1).astype(np.int64) - first
    ids = np.where((ids >= 0) & (ids < experts), ids, experts)
    slots = np.argsort(ids, kind="stable")
    count = np.bincount(ids, minlength=experts + 1)[:experts]
    offsets = np.concatenate([[0], np.cumsum((count + pad - 1) // pad * pad)])
    order = np.full(rows, -1)
    pos = np.full(len(ids), -1)
    start = 0
    for e in range(experts):
        mine = slots[start:start + count[e]]
        order[offsets[e]:offsets[e] + count[e]] = mine
        pos[mine] = offsets[e] + np.arange(count[e])
        start += count[e]
    return offsets, order, pos


def sort(ids, first, experts, pad, extra=0, stream=None):
    """The GPU's sort of a numpy array of ids, with what surrounds its outputs checked."""
    tokens, k = ids.shape
    rows = hr.hr_experts_rows(tokens, k, experts, pad) + extra
    frames = [torch.full((n + 16,), 77, dtype=torch.int32, device=DEV) for n in (experts + 1, rows, tokens * k)]
    offsets, order = frames[0][8:8 + experts + 1], frames[1][8:8 + rows]
    pos = frames[2][8:8 + tokens * k].view(tokens, k)
    need = hr.hr_experts_sort_workspace(tokens, k, experts)
    ws = torch.full((need + 32,), 255, dtype=torch.uint8, device=DEV)[:need] if need else None
    hr.experts_sort(torch.from_numpy(ids.astype(np.int32)).to(DEV), offsets, order, pos, first=first, pad=pad,
                    workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for f in frames:
        assert (f[:8] == 77).all() and (f[-8:] == 77).all(), "written outside an output"
    return offsets, order, pos


def check_sort(ids, first, experts, pad, extra=0):
    print(f"sort {ids.shape} of {experts} from {first}, pad {pad}", flush=True)
    got = sort(ids, first, experts, pad, extra)
    want = sort_reference(ids, first, experts, pad, got[1].numel())
    for name, g, w in zip(("offsets", "order", "pos"), got, want):
        np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), w, err_msg=name)
    return got


def picks(seed, tokens, k, experts, drop=0.0):
    rng = np.random.default_rng(seed)
    liked = rng.standard_normal((tokens, experts)) + rng.standard_normal(experts)
    ids = np.argsort(-liked, axis=1)[:, :k].astype(np.int64)
    ids[rng.random(tokens) < drop] = -1
    return ids


# tokens and k on both sides of what one workgroup sorts (8192 slots) and of
# a chunk and a wave of the many
@pytest.mark.parametrize("tokens,k,experts", [
    (1, 1, 1), (1, 8, 8), (3, 2, 5), (64, 6, 64), (65, 8, 128), (1024, 8, 128), (1025, 8, 128), (2731, 3, 60),
    (8193, 1, 2), (4096, 4, 512), (5000, 7, 513), (700, 10, 1024), (9999, 10, 1024), (66000, 8, 256), (300, 32, 64),
    (1 << 20, 1, 16)])
@pytest.mark.parametrize("pad", [1, 16])
def test_sort(tokens, k, experts, pad):
    if tokens * experts <= 1 << 24:
        ids = picks(tokens, tokens, k, experts, 0.03)
    else:
        ids = np.random.default_rng(tokens).integers(-1, experts, (tokens, k))
    check_sort(ids, 0, experts, pad)


# both sides of one, two and eight slots of a thread, and shares of a wave above
# what it keeps: up to 512 experts a workgroup has 1024 threads, beyond them 512
@pytest.mark.parametrize("slots,experts", [
    (256, 384), (257, 384), (512, 600), (513, 600), (1024, 40), (1025, 40), (1024, 600), (1025, 600), (2048, 40),
    (2049, 40), (4096, 600), (4097, 600), (8192, 600), (8192, 40), (525000, 40), (525000, 600), (1100000, 600),
    (2200000, 40)])
def test_sort_shares(slots, experts):
    ids = np.random.default_rng(slots).integers(-1, experts + 2, (slots, 1))
    check_sort(ids, 0, experts, 16)
    ids[:] = experts - 1                                        # one expert takes all
    check_sort(ids, 0, experts, 3)


# few and many sorted rows: one to eight of them to the same lanes
@pytest.mark.parametrize("tokens,k,experts,pad", [(9, 3, 384, 16), (900, 4, 60, 64), (3000, 6, 500, 40),
                                                  (9000, 7, 512, 16)])
@pytest.mark.parametrize("width", [64, 200, 1100])
def test_padding_is_zero(tokens, k, experts, pad, width):
    offsets, order, pos, o, ph, used = buffers(tokens, tokens, k, experts, pad)
    m = Maker(width)
    x = m.normal(tokens, width, dtype=torch.float16)
    out = m.place(len(o), width, torch.float16, width + 4, 2)
    print(f"padding {tokens}x{width} k={k} experts={experts} pad={pad}", flush=True)
    hr.experts_gather(x.to(DEV), pos, out, offsets=offsets, order=order)
    torch.cuda.synchronize()
    want = torch.full((len(o), width), 7.0).half()
    want[:used] = 0
    want[torch.from_numpy(o >= 0)] = x[torch.from_numpy(o[o >= 0] // k)]
    assert torch.equal(out.cpu(), want)
    m.check_frames()
    run_grad(m, torch.float16, tokens, width, k, pos, ph, offsets, order, o, weights=torch.rand(tokens, k, generator=m.g),
             used=used)


@pytest.mark.parametrize("tokens", [700, 40000])
def test_sort_of_a_rank(tokens):
    """A rank's share of the experts, every id outside it of any value."""
    ids = picks(1, tokens, 4, 96)
    ids[::7, 1] = -(1 << 31)
    ids[::5, 2] = (1 << 31) - 1
    for first, experts, pad in ((0, 24, 1), (24, 24, 128), (72, 24, 7), (95, 1, 64), (96, 5, 16)):
        check_sort(ids, first, experts, pad)


@pytest.mark.parametrize("tokens", [500, 50000])
def test_sort_skewed(tokens):
    for ids in (np.full((tokens, 2), 3), np.full((tokens, 2), -1), np.tile([[0, 63]], (tokens, 1)),
                np.repeat(np.arange(tokens)[:, None] % 64, 2, 1)):
        check_sort(ids, 0, 64, 32, extra=1000)


def test_sort_nothing():
    offsets, order, _ = sort(np.zeros((0, 4), dtype=np.int64), 0, 16, 8, extra=100)
    assert (offsets == 0).all() and (order == -1).all()


def test_rows_and_workspace_sizes():
    assert hr.hr_experts_rows(10, 4, 64, 1) == 40
    assert hr.hr_experts_rows(10, 4, 64, 16) == 40 + 40 * 15      # at most one segment per slot
    assert hr.hr_experts_rows(1000, 4, 64, 16) == 4000 + 64 * 15


def buffers(seed, tokens, k, experts, pad, drop=0.05, first=0, local=None):
    ids = picks(seed, tokens, k, experts, drop if tokens > 4 else 0.0)
    offsets, order, pos = sort(ids, first, local or experts, pad)
    return offsets, order, pos, order.cpu().numpy(), pos.cpu().numpy(), int(offsets[-1])


WIDTHS = [1, 7, 8, 9, 100, 128, 129, 511, 512, 513, 2047, 2048, 2049, 4096, 5121]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["f16", "bytes", "e4m3+scales"])
def test_gather(width, kind):
    tokens, k, experts, pad = 67, 5, 12, 8
    offsets, order, pos, o, _, used = buffers(width, tokens, k, experts, pad)
    m = Maker(width)
    if kind == "f16":
        x = m.normal(tokens, width, dtype=torch.float16)
    else:
        x = torch.randint(0, 256, (tokens, width), generator=m.g, dtype=torch.uint8)
    groups = -(-width // 128)
    s = torch.rand(tokens, groups, generator=m.g) if kind == "e4m3+scales" else None
    for stride, offset in ((None, 0), (width + 3, 1)):
        print(f"gather {kind} width {width} stride {stride}", flush=True)
        dx = m.place(tokens, width, x.dtype, stride, offset, x)
        out = m.place(len(o), width, x.dtype, stride, offset)
        ds = m.place(tokens, groups, torch.float32, groups + 1, 1, s) if s is not None else None
        so = m.place(len(o), groups, torch.float32, groups + 2, 3) if s is not None else None
        f8 = torch.float8_e4m3fn
        hr.experts_gather(dx.view(f8) if s is not None else dx, pos, out.view(f8) if s is not None else out,
                          offsets=offsets, order=order, scales=ds, scales_out=so)
        torch.cuda.synchronize()
        for src, got, fill in ((x, out, 7), (s, so, 7.0)):
            if src is None:
                continue
            want = torch.full((len(o), src.shape[1]), fill).to(src.dtype)
            want[:used] = 0
            here = torch.from_numpy(o >= 0)
            want[here] = src[torch.from_numpy(o[o >= 0] // k)]
            assert torch.equal(got.cpu(), want), kind
        m.check_frames()


def test_gather_leaves_padding_alone_without_order():
    offsets, order, pos, o, _, used = buffers(3, 50, 4, 8, 16)
    x = torch.randn(50, 256, device=DEV).half()
    out = torch.full((len(o), 256), 5.0, dtype=torch.float16, device=DEV)
    hr.experts_gather(x, pos, out)
    here = torch.from_numpy(o >= 0).to(DEV)
    assert (out[~here] == 5).all()
    assert torch.equal(out[here], x[torch.from_numpy(o[o >= 0] // 4).to(DEV)])


def combine_reference(z, pos, w, addend, hidden):
    """(sum, sum of magnitudes) in 64 bits."""
    tokens, k = pos.shape
    y = torch.zeros(tokens, hidden, dtype=torch.float64) if addend is None else addend.double()
    size = y.abs()
    for j in range(k):
        t = torch.from_numpy(np.flatnonzero((pos[:, j] >= 0) & (pos[:, j] < len(z))))
        p = torch.from_numpy(pos[:, j])[t].long()
        term = z[p].double() * (w[t, j, None].double() if w is not None else 1.0)
        y[t] += term
        size[t] += term.abs()
    return y, size


def sum_bound(dtype, ref, size, k):
    """k multiply-adds (and the addend) in binary32, then one rounding."""
    return half_step(dtype, ref) * (1 + 2.0 ** -8) + size * (k + 2) * F32


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_combine(dt, hidden):
    dtype = TYPES[dt]
    tokens, k, experts, pad = 67, 6, 12, 8
    _, _, pos, o, ph, _ = buffers(hidden, tokens, k, experts, pad)
    m = Maker(hidden)
    z = m.normal(len(o), hidden, dtype=dtype)
    z[torch.from_numpy(o < 0)] = float("nan")                    # rows of no slot are not read
    w, add = torch.rand(tokens, k, generator=m.g), m.normal(tokens, hidden, dtype=dtype)
    w[torch.from_numpy(ph < 0)] = float("inf")                   # nor are their weights
    for weights, addend, stride, offset in ((w, None, None, 0), (None, add, hidden + 5, 1), (w, add, hidden + 8, 3),
                                            (w, "in place", hidden + 1, 0)):
        print(f"combine {dt} {hidden} stride {stride} addend {addend is not None}", flush=True)
        dz = m.place(len(o), hidden, dtype, stride, offset, z)
        da = m.place(tokens, hidden, dtype, stride, offset, add) if addend is not None else None
        out = da if isinstance(addend, str) else m.place(tokens, hidden, dtype, stride, offset + 1)
        hr.experts_combine(dz, pos, out, weights=weights.to(DEV) if weights is not None else None, addend=da)
        torch.cuda.synchronize()
        ref, size = combine_reference(z, ph, weights, add if addend is not None else None, hidden)
        within(out, ref, sum_bound(dtype, ref, size, k), "combine")
        m.check_frames()


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("tokens", [1, 2, 333])
def test_combine_picks(k, tokens):
    dtype = torch.bfloat16
    for hidden in (64, 1000, 4104):
        _, _, pos, o, ph, _ = buffers(k, tokens, k, 40, 1)
        m = Maker(k)
        z, w = m.normal(len(o), hidden, dtype=dtype), torch.rand(tokens, k, generator=m.g)
        out = torch.empty(tokens, hidden, dtype=dtype, device=DEV)
        hr.experts_combine(z.to(DEV), pos, out, weights=w.to(DEV))
        ref, size = combine_reference(z, ph, w, None, hidden)
        within(out, ref, sum_bound(dtype, ref, size, k), "combine")
        run_grad(m, dtype, tokens, hidden, k, pos, ph, None, None, o, weights=w)


def run_grad(m, dtype, tokens, hidden, k, pos, ph, offsets, order, o, weights=None, stride=None, offset=0, used=None,
             in_place=False, want=("dz", "dw")):
    dy, z = m.normal(tokens, hidden, dtype=dtype), m.normal(len(o), hidden, dtype=dtype)
    ddy = m.place(tokens, hidden, dtype, stride, offset, dy)
    dzz = m.place(len(o), hidden, dtype, stride, offset + 1, z)
    dz = dzz if in_place else m.place(len(o), hidden, dtype, stride, offset)
    dw = torch.full((tokens, k), 9.0, device=DEV)
    hr.experts_combine_grad(ddy, dzz, pos, weights.to(DEV) if weights is not None else None,
                            dz if "dz" in want else None, dw if "dw" in want else None, offsets=offsets, order=order)
    torch.cuda.synchronize()
    ref = (z if in_place else torch.full((len(o), hidden), 7.0).to(dtype)).double()
    dots, size = torch.zeros(tokens, k, dtype=torch.float64), torch.zeros(tokens, k, dtype=torch.float64)
    if order is not None:
        ref[:used] = 0
    exact = torch.ones(len(o), dtype=torch.bool)
    for j in range(k):
        t = torch.from_numpy(np.flatnonzero(ph[:, j] >= 0))
        p = torch.from_numpy(ph[:, j])[t].long()
        exact[p] = False
        ref[p] = dy[t].double() * (weights[t, j, None].double() if weights is not None else 1.0)
        prod = dy[t].double() * z[p].double()
        dots[t, j], size[t, j] = prod.sum(1), prod.abs().sum(1)
    if "dz" in want:
        # a product of 16 and 24 bits rounded to binary32, then to the type
        tol = half_step(dtype, ref) * (1 + 2.0 ** -8) + ref.abs() * F32
        tol[exact] = 0
        within(dz, ref, tol, "dz")
    if "dw" in want:
        # a lane's terms in sequence, then the tree: at most hidden / 16 + 10 additions
        within(dw, dots, size * (hidden / 16 + 32) * F32, "dweights")
    m.check_frames()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden", WIDTHS)
def test_combine_grad(dt, hidden):
    tokens, k, experts, pad = 45, 5, 12, 8
    offsets, order, pos, o, ph, used = buffers(hidden, tokens, k, experts, pad)
    m = Maker(hidden)
    w = torch.rand(tokens, k, generator=m.g)
    for weights, stride, offset, ordered, in_place in ((w, None, 0, True, False), (None, hidden + 3, 1, False, False),
                                                       (w, hidden + 1, 2, True, True)):
        print(f"combine grad {dt} {hidden} stride {stride} ordered {ordered} in place {in_place}", flush=True)
        run_grad(m, TYPES[dt], tokens, hidden, k, pos, ph, offsets if ordered else None, order if ordered else None,
                 o, weights, stride, offset, used, in_place)
    run_grad(m, TYPES[dt], tokens, hidden, k, pos, ph, None, None, o, w, want=("dz",))
    run_grad(m, TYPES[dt], tokens, hidden, k, pos, ph, None, None, o, w, want=("dw",))


def test_gather_gradient_is_the_combine():
    """<gather(x), g> and <x, combine(g)> agree: the one is the other's transpose."""
    tokens, k, hidden = 200, 4, 640
    offsets, order, pos, o, ph, used = buffers(9, tokens, k, 16, 16)
    m = Maker(9)
    x, g = m.normal(tokens, hidden, dtype=torch.float16), m.normal(len(o), hidden, dtype=torch.float16)
    out = torch.zeros(len(o), hidden, dtype=torch.float16, device=DEV)
    hr.experts_gather(x.to(DEV), pos, out, offsets=offsets, order=order)
    dx = torch.empty(tokens, hidden, dtype=torch.float16, device=DEV)
    hr.experts_combine(g.to(DEV), pos, dx)
    left, right = (out.cpu().double() * g.double()).sum(), (x.double() * dx.cpu().double()).sum()
    size = (x.double().abs() * dx.cpu().double().abs()).sum()
    # dx is rounded to binary16 once, 2^-11 of each value at most
    assert abs(left - right) <= size * 2.0 ** -11


def test_grad_against_differences():
    """dz and dweights against central differences of the combine in 64 bits
    (linear in each, so a difference is exact but for its own roundings)."""
    tokens, k, hidden, step = 3, 2, 10, 1.0
    _, _, pos, o, ph, _ = buffers(4, tokens, k, 4, 1, drop=0.0)
    m = Maker(4)
    dy, z = m.normal(tokens, hidden, dtype=torch.float16), m.normal(len(o), hidden, dtype=torch.float16)
    w = torch.rand(tokens, k, generator=m.g)

    def loss(z, w):
        y = torch.zeros(tokens, hidden, dtype=torch.float64)
        for t in range(tokens):
            for j in range(k):
                y[t] += w[t, j] * z[ph[t, j]]
        return (y * dy.double()).sum()

    zref, wref = torch.zeros(len(o), hidden).double(), torch.zeros(tokens, k).double()
    for i in np.ndindex(len(o), hidden):
        e = torch.zeros(len(o), hidden).double()
        e[i] = step
        zref[i] = (loss(z.double() + e, w.double()) - loss(z.double() - e, w.double())) / (2 * step)
    for i in np.ndindex(tokens, k):
        e = torch.zeros(tokens, k).double()
        e[i] = step
        wref[i] = (loss(z.double(), w.double() + e) - loss(z.double(), w.double() - e)) / (2 * step)
    dz, dw = torch.empty(len(o), hidden, dtype=torch.float16, device=DEV), torch.empty(tokens, k, device=DEV)
    hr.experts_combine_grad(dy.to(DEV), z.to(DEV), pos, w.to(DEV), dz, dw)
    within(dz, zref, half_step(torch.float16, zref) * (1 + 2.0 ** -8) + zref.abs() * F32 + 1e-12, "dz")
    within(dw, wref, torch.full_like(wref, hidden * 9 * 32 * F32), "dweights")


@pytest.mark.parametrize("hidden", [9, 513, 1001, 2049])
def test_grad_in_place_with_overflow(hidden):
    """dz over z, dz beyond binary16's range: dweights are of z as it was."""
    tokens, k = 40, 3
    _, _, pos, o, ph, _ = buffers(hidden, tokens, k, 6, 1, drop=0.0)
    m = Maker(hidden)
    z, dy = m.normal(len(o), hidden, dtype=torch.float16), m.normal(tokens, hidden, sigma=2000.0, dtype=torch.float16)
    w = torch.full((tokens, k), 1000.0)
    dz, dw = z.to(DEV), torch.empty(tokens, k, device=DEV)
    hr.experts_combine_grad(dy.to(DEV), dz, pos, w.to(DEV), dz, dw)
    torch.cuda.synchronize()
    assert torch.isinf(dz).any()
    prod = dy.double()[:, None] * z.double()[torch.from_numpy(ph).long()]
    within(dw, prod.sum(2), prod.abs().sum(2) * (hidden / 16 + 32) * F32, "dweights")


def test_foreign_rows_are_left_out():
    """A pos outside the buffer is no row: nothing is read or written there."""
    pos = torch.tensor([[0, 5], [-1, 2], [-(1 << 31), (1 << 31) - 1]], dtype=torch.int32)
    z, w = torch.randn(4, 64).half(), torch.rand(3, 2)
    frame = torch.full((8, 64), 7.0, dtype=torch.float16, device=DEV)
    out = torch.empty(3, 64, dtype=torch.float16, device=DEV)
    hr.experts_combine(z.to(DEV), pos.to(DEV), out, weights=w.to(DEV))
    ref, size = combine_reference(z, pos.numpy(), w, None, 64)
    within(out, ref, sum_bound(torch.float16, ref, size, 2), "combine")
    x = torch.randn(3, 64, device=DEV).half()
    hr.experts_gather(x, pos.to(DEV), frame[2:6])
    dw = torch.empty(3, 2, device=DEV)
    hr.experts_combine_grad(x, z.to(DEV), pos.to(DEV), w.to(DEV), None, dw)
    torch.cuda.synchronize()
    assert (frame[:2] == 7).all() and (frame[6:] == 7).all()
    assert torch.equal(frame[2], x[0]) and torch.equal(frame[4], x[1]) and (frame[3] == 7).all()
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and (dw[2] == 0).all() and dw[0, 0] != 0


def test_rows_past_four_gib():
    """Sorted rows past 2^32 bytes and 2^31 values: gathered, combined and back."""
    tokens, k, hidden = 17000, 8, 16384
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    ids = np.random.default_rng(0).integers(0, 32, (tokens, k))
    offsets, order, pos = sort(ids, 0, 32, 1)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    big = torch.empty(tokens * k, hidden, dtype=torch.bfloat16, device=DEV)
    assert big.numel() > 1 << 31
    hr.experts_gather(x, pos, big, offsets=offsets, order=order)
    token = torch.div(order, k, rounding_mode="floor").long()
    for a in range(0, tokens * k, 20000):
        assert torch.equal(big[a:a + 20000], x[token[a:a + 20000]])
    out = torch.empty_like(x)
    w = torch.full((tokens, k), 0.125, device=DEV)
    hr.experts_combine(big, pos, out, weights=w)                 # eight eighths of every row
    assert torch.equal(out, x)
    dw = torch.empty(tokens, k, device=DEV)
    hr.experts_combine_grad(x, big, pos, w, big, dw)
    assert torch.equal(big[-3000:].float(), x[token[-3000:]].float() * 0.125)
    ref = x.double().square().sum(1, keepdim=True)
    assert ((dw.double() - ref).abs() <= ref * (hidden / 16 + 32) * F32).all()


def test_repeats_streams_and_graphs():
    tokens, k, experts, hidden, pad = 3000, 4, 32, 1024, 16
    m = Maker(5)
    ids = torch.empty(tokens, k, dtype=torch.int32, device=DEV)
    offsets, order, pos = hr.experts_buffers(tokens, k, experts, pad)
    ws = torch.empty(hr.hr_experts_sort_workspace(tokens, k, experts), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    x, out, dy = (m.normal(tokens, hidden, dtype=torch.float16).to(DEV) for _ in range(3))
    s, dz = (torch.zeros(order.numel(), hidden, dtype=torch.float16, device=DEV) for _ in range(2))
    w, dw = torch.rand(tokens, k, device=DEV), torch.empty(tokens, k, device=DEV)
    outs = (offsets, order, pos, s, out, dz, dw)

    def step(stream=None, workspace=ws):
        hr.experts_sort(ids, offsets, order, pos, pad=pad, workspace=workspace, stream=stream)
        hr.experts_gather(x, pos, s, offsets=offsets, order=order, stream=stream)
        hr.experts_combine(s, pos, out, weights=w, stream=stream)
        hr.experts_combine_grad(dy, s, pos, w, dz, dw, offsets=offsets, order=order, stream=stream)

    def new(seed):
        ids.copy_(torch.from_numpy(picks(seed, tokens, k, experts, 0.1).astype(np.int32)))

    new(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    for seed in range(1, 4):
        new(seed)
        for t in outs:
            t.zero_()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for again in (graph.replay, lambda: step(other, None), step):
            for t in outs:
                t.zero_()
            torch.cuda.synchronize()
            again()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, outs)), seed


def test_binding_refusals():
    ids = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    offsets, order, pos = hr.experts_buffers(8, 2, 4)
    x, s = torch.zeros(8, 64, dtype=torch.float16, device=DEV), torch.zeros(16, 64, dtype=torch.float16, device=DEV)
    w = torch.ones(8, 2, device=DEV)
    for bad, err in [(lambda: hr.experts_sort(ids.long(), offsets, order, pos), TypeError),
                     (lambda: hr.experts_sort(ids.cpu(), offsets, order, pos), TypeError),
                     (lambda: hr.experts_sort(ids.view(-1), offsets, order, pos), ValueError),
                     (lambda: hr.experts_sort(ids, offsets, order, pos[:7]), ValueError),
                     (lambda: hr.experts_sort(ids, offsets, order[:15], pos), hr.HrError),
                     (lambda: hr.experts_sort(ids, offsets, order, pos, pad=2), hr.HrError),
                     (lambda: hr.experts_sort(ids, offsets, order, pos, first=-1), hr.HrError),
                     (lambda: hr.experts_gather(x, pos, s.bfloat16()), TypeError),
                     (lambda: hr.experts_gather(x, pos, s[:, :32]), ValueError),
                     (lambda: hr.experts_gather(x, pos[:7], s), ValueError),
                     (lambda: hr.experts_gather(x, pos, s, order=order), ValueError),
                     (lambda: hr.experts_gather(x, pos, s, scales=w), ValueError),
                     (lambda: hr.experts_gather(x, pos, s, order=order[:9], offsets=offsets), ValueError),
                     (lambda: hr.experts_combine(s.float(), pos, x), TypeError),
                     (lambda: hr.experts_combine(s, pos, x.float()), TypeError),
                     (lambda: hr.experts_combine(s, pos, x, weights=w.half()), TypeError),
                     (lambda: hr.experts_combine(s, pos, x, weights=w[:, :1]), ValueError),
                     (lambda: hr.experts_combine(s, pos, s[:8]), hr.HrError),
                     (lambda: hr.experts_combine(s, pos.long(), x), TypeError),
                     (lambda: hr.experts_combine_grad(x, s, pos, w), hr.HrError),
                     (lambda: hr.experts_combine_grad(x, s, pos, w, s[1:], None), ValueError),
                     (lambda: hr.experts_combine_grad(x, s, pos, w, None, w.double()), TypeError)]:
        with pytest.raises(err):
            bad()
    ids[:, 1] = 3
    hr.experts_sort(ids, offsets, order, pos)
    assert offsets.cpu().tolist() == [0, 8, 8, 8, 16] and order.cpu().tolist() == [*range(0, 16, 2), *range(1, 16, 2)]


# a rank's share of the experts in buffers of the rows that it uses: fewer than
# tokens x k, none to spare, a few, and as many as there are slots
@pytest.mark.parametrize("tokens,k,experts,first,local,pad", [(11, 3, 12, 5, 2, 4), (64, 6, 64, 16, 16, 16),
                                                              (500, 8, 64, 56, 8, 16), (3000, 4, 128, 0, 16, 64)])
@pytest.mark.parametrize("width", [64, 300, 1100])
def test_padding_is_zero_in_a_trimmed_buffer(tokens, k, experts, first, local, pad, width):
    offsets, order, pos, o, ph, used = buffers(tokens, tokens, k, experts, pad, first=first, local=local)
    assert used < tokens * k and (o[:used] < 0).any()
    m = Maker(width)
    groups = -(-width // 128)
    x, codes = m.normal(tokens, width, dtype=torch.float16), torch.randint(0, 256, (tokens, width), generator=m.g,
                                                                           dtype=torch.uint8)
    s = torch.rand(tokens, groups, generator=m.g)
    for n in (used, min(used + 3, tokens * k), tokens * k):
        print(f"trimmed {tokens}x{width} k={k} pad={pad}: {n} rows, {used} used", flush=True)
        part, of = order[:n], torch.from_numpy(o[:n])
        for src, scales in ((x, None), (codes, s)):
            out = m.place(n, width, src.dtype, width + 2, 1)
            so = m.place(n, groups, torch.float32, groups + 1, 1) if scales is not None else None
            hr.experts_gather(src.to(DEV), pos, out, offsets=offsets, order=part,
                              scales=scales.to(DEV) if scales is not None else None, scales_out=so)
            torch.cuda.synchronize()
            for a, got in ((src, out), (scales, so)):
                if a is None:
                    continue
                want = torch.full((n, a.shape[1]), 7).to(a.dtype)
                want[:used] = 0
                want[of >= 0] = a[of[of >= 0] // k]
                assert torch.equal(got.cpu(), want), f"{a.dtype}, {n} rows"
        for in_place in (False, True):
            run_grad(m, torch.bfloat16, tokens, width, k, pos, ph, offsets, part, o[:n],
                     weights=torch.rand(tokens, k, generator=m.g), used=used, in_place=in_place)
    m.check_frames()


def test_gather_takes_the_scales_of_rows():
    """A scale per row in one dimension, as reduce_rmsnorm writes it."""
    tokens, k, hidden = 20, 3, 512
    offsets, order, pos, o, _, used = buffers(7, tokens, k, 6, 4)
    h = Maker(7).normal(tokens, hidden, dtype=torch.float16).to(DEV)
    f8 = torch.float8_e4m3fn
    codes, scales = torch.empty(tokens, hidden, dtype=f8, device=DEV), torch.empty(tokens, device=DEV)
    hr.reduce_rmsnorm([h], out8=codes, scales=scales)
    out, scales_out = torch.empty(len(o), hidden, dtype=f8, device=DEV), torch.full((len(o),), 7.0, device=DEV)
    hr.experts_gather(codes, pos, out, offsets=offsets, order=order, scales=scales, scales_out=scales_out)
    torch.cuda.synchronize()
    want = torch.full((len(o),), 7.0)
    want[:used] = 0
    want[torch.from_numpy(o >= 0)] = scales.cpu()[torch.from_numpy(o[o >= 0] // k)]
    assert torch.equal(scales_out.cpu(), want)
    here = torch.from_numpy(o >= 0).to(DEV)
    assert torch.equal(out.view(torch.uint8)[here], codes.view(torch.uint8)[torch.from_numpy(o[o >= 0] // k).to(DEV)])
    with pytest.raises(ValueError):
        hr.experts_gather(codes, pos, out, offsets=offsets, order=order, scales=scales[:-1], scales_out=scales_out)
    with pytest.raises(ValueError):
        hr.experts_gather(codes, pos, out, offsets=offsets, order=order, scales=scales, scales_out=scales_out[1:])
    # and one dimension for the scales of a single row stays what it was
    row, one = torch.rand(4, device=DEV), torch.zeros(4, device=DEV)
    hr.experts_gather(codes[:1], torch.zeros(1, 1, dtype=torch.int32, device=DEV), out[:1], scales=row, scales_out=one)
    assert torch.equal(row, one) and torch.equal(out[0].view(torch.uint8), codes[0].view(torch.uint8))


# rows of 64 MiB or more pass the caches by: both sides of every number of lanes,
# two units of a lane (2304), whole units and odd lengths
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hidden", [100, 128, 129, 500, 512, 1000, 2047, 2303, 2304, 4097])
def test_streamed_rows(dt, hidden):
    """Large calls give the bits of calls on parts of the tokens, and leave what
    lies around their rows alone."""
    dtype, g, k, experts, pad = TYPES[dt], torch.Generator(device=DEV).manual_seed(hidden), 3, 40, 16
    tokens = (1 << 26) // (hidden * 2 * k) + 5
    ids = np.random.default_rng(hidden).integers(-1, experts, (tokens, k))
    offsets, order, pos = sort(ids, 0, experts, pad)
    rows = order.numel()
    print(f"streamed experts {dt} {tokens}x{hidden}, {rows} rows", flush=True)

    def buffer(n, value=None):
        b = torch.empty(1 + n * (hidden + 3) + 8, dtype=dtype, device=DEV)
        b = b.normal_(generator=g) if value is None else b.fill_(value)
        return b, lambda b, a=0, e=n: b.as_strided((e - a, hidden), (hidden + 3, 1), 1 + a * (hidden + 3))

    (x, of_tokens), (add, _) = buffer(tokens), buffer(tokens)
    z, of_rows = buffer(rows)
    w = torch.rand(tokens, k, generator=g, device=DEV)
    whole, cuts = [(0, tokens)], [tokens * i // 4 for i in range(5)]
    got = []
    for parts in (whole, list(zip(cuts, cuts[1:]))):
        s, dz, over = buffer(rows, 7)[0], buffer(rows, 7)[0], z.clone()
        y, plus, dx = buffer(tokens, 7)[0], add.clone(), buffer(tokens, 7)[0]
        dw, dw2 = (torch.full((tokens, k), 7.0, device=DEV) for _ in range(2))
        for a, b in parts:
            p = pos[a:b]
            hr.experts_gather(of_tokens(x, a, b), p, of_rows(s), offsets=offsets, order=order)
            hr.experts_combine(of_rows(z), p, of_tokens(y, a, b), weights=w[a:b])
            hr.experts_combine(of_rows(z), p, of_tokens(plus, a, b), weights=w[a:b], addend=of_tokens(plus, a, b))
            hr.experts_combine(of_rows(z), p, of_tokens(dx, a, b))
            hr.experts_combine_grad(of_tokens(x, a, b), of_rows(z), p, w[a:b], of_rows(dz), dw[a:b], offsets=offsets,
                                    order=order)
            hr.experts_combine_grad(of_tokens(x, a, b), of_rows(over), p, w[a:b], of_rows(over), dw2[a:b])
        torch.cuda.synchronize()
        assert torch.equal(dw, dw2)
        got.append((s, y, plus, dx, dz, dw, over))
    for name, a, b in zip(("gather", "combine", "addend in place", "no weights", "dz", "dweights", "dz in place"), *got):
        bad = a.view(torch.uint8) != b.view(torch.uint8)
        assert not bad.any(), f"{name}: {int(bad.sum())} bytes differ"
    used = int(offsets[-1])
    assert (of_rows(got[0][0])[:used][order[:used] < 0] == 0).all() and (of_rows(got[0][0])[used:] == 7).all()
