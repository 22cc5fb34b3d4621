"""GPU: gated experts put together from the operators, as a layer uses them:
sorted, gathered, multiplied, activated, multiplied and combined, in 16 bits
forward and backward and in e4m3, and captured into a graph."""
import pytest
import torch

from _gpu import needs_gpu
from _products import F8, wide_blocks, wide_rows
from message_fp16_all_amd import hr

pytestmark = [pytest.mark.gpu, needs_gpu]
DEV = "cuda:0"


def rel(got, ref):
    return float((got.detach().cpu().double() - ref).norm() / ref.norm())


class Mlp:
    """experts gated MLPs of hidden -> inner -> hidden over k picks of every token."""

    def __init__(self, tokens, hidden, inner, experts, k, dt, pad=1, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(tokens, hidden, generator=g).to(dt).to(DEV)
        self.up = (torch.randn(experts, 2 * inner, hidden, generator=g) / hidden ** 0.5).to(dt).to(DEV)
        self.down = (torch.randn(experts, hidden, inner, generator=g) / inner ** 0.5).to(dt).to(DEV)
        self.ids = torch.stack([torch.randperm(experts, generator=g)[:k] for _ in range(tokens)]).to(torch.int32).to(DEV)
        self.weights = torch.rand(tokens, k, generator=g).to(DEV)
        self.dy = torch.randn(tokens, hidden, generator=g).to(dt).to(DEV)
        self.offsets, self.order, self.pos = hr.experts_buffers(tokens, k, experts, pad)
        self.pad, rows = pad, self.order.numel()

        def new(width, dtype=dt, n=rows):
            return torch.empty(n, width, dtype=dtype, device=DEV)

        self.new = new
        self.rows, self.h, self.a, self.z = new(hidden), new(2 * inner), new(inner), new(hidden)
        self.y, self.dx = new(hidden, n=tokens), new(hidden, n=tokens)
        self.dz, self.da, self.drows = new(hidden), new(inner), new(hidden)
        self.dup, self.ddown = torch.empty_like(self.up), torch.empty_like(self.down)
        self.dweights = torch.empty_like(self.weights)

    def forward(self):
        hr.experts_sort(self.ids, self.offsets, self.order, self.pos, pad=self.pad)
        hr.experts_gather(self.x, self.pos, self.rows, offsets=self.offsets, order=self.order)
        hr.experts_product(self.rows, self.up, self.h, offsets=self.offsets)
        hr.experts_act(self.h, self.a, offsets=self.offsets)
        hr.experts_product(self.a, self.down, self.z, offsets=self.offsets)
        return hr.experts_combine(self.z, self.pos, self.y, weights=self.weights)

    def backward(self):
        hr.experts_combine_grad(self.dy, self.z, self.pos, self.weights, self.dz, self.dweights, offsets=self.offsets,
                                order=self.order)
        hr.experts_product(self.dz, self.down, self.da, offsets=self.offsets, transposed=True)
        hr.experts_product_grad(self.dz, self.a, self.ddown, offsets=self.offsets)
        hr.experts_act_grad(self.da, self.h, self.h, offsets=self.offsets)
        hr.experts_product(self.h, self.up, self.drows, offsets=self.offsets, transposed=True)
        hr.experts_product_grad(self.h, self.rows, self.dup, offsets=self.offsets)
        return hr.experts_combine(self.drows, self.pos, self.dx)

    def reference(self, up=None, down=None):
        """(y, gradients) in 64 bits with autograd."""
        leaf = [t.cpu().double().requires_grad_() for t in
                (self.x, self.up if up is None else up, self.down if down is None else down, self.weights)]
        x, up, down, weights = leaf
        y = torch.zeros_like(x)
        ids = self.ids.cpu().long()
        inner = down.shape[2]
        for e in range(up.shape[0]):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            h = x[t] @ up[e].t()
            a = torch.nn.functional.silu(h[:, :inner]) * h[:, inner:]
            y = y.index_add(0, t, (a @ down[e].t()) * weights[t, j, None])
        (y * self.dy.cpu().double()).sum().backward()
        return y.detach(), dict(zip(("dx", "dup", "ddown", "dweights"), (t.grad for t in leaf)))


SIZES = [(1, 64, 32, 4, 2, 1), (37, 256, 96, 8, 3, 16), (300, 200, 136, 6, 2, 1), (500, 264, 72, 3, 3, 64)]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,hidden,inner,experts,k,pad", SIZES)
def test_forward_and_backward(dt, tokens, hidden, inner, experts, k, pad):
    m = Mlp(tokens, hidden, inner, experts, k, dt, pad, seed=tokens)
    m.forward()
    m.backward()
    torch.cuda.synchronize()
    y, grads = m.reference()
    half = torch.finfo(dt).eps / 2
    # forward rounds h (which shifts gate and up), a, z and y; backward dz, da, the
    # two halves of dh on the rounded h, drows and dx
    assert rel(m.y, y) <= 5 * half
    for name, ref in grads.items():
        assert rel(getattr(m, name), ref) <= 10 * half, name


def test_captured():
    """Graphs replayed with other tokens and picks give what eager calls give."""
    a, b = (Mlp(64, 256, 128, 8, 2, torch.bfloat16, seed=1) for _ in range(2))
    a.forward()
    a.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward()
        a.backward()
    for i in range(3):
        other = Mlp(64, 256, 128, 8, 2, torch.bfloat16, seed=10 + i)
        for name in ("x", "ids", "dy", "up"):
            getattr(a, name).copy_(getattr(other, name))
            getattr(b, name).copy_(getattr(other, name))
        graph.replay()
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        for name in ("y", "dx", "dup", "ddown", "dweights"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name


def blocks(w):
    """(codes, scales) of matrices with a scale per 128 x 128 values."""
    e, r, c = w.shape
    nr, nc = -(-r // 128), -(-c // 128)
    full = torch.zeros(e, nr * 128, nc * 128)
    full[:, :r, :c] = w.float().cpu()
    scales = full.view(e, nr, 128, nc, 128).abs().amax((2, 4)) / 448 + 1e-30
    wide = scales.repeat_interleave(128, 1).repeat_interleave(128, 2)
    return (full / wide)[:, :r, :c].contiguous().to(F8), scales


@pytest.mark.parametrize("tokens,hidden,inner,experts,k", [(1, 256, 128, 4, 2), (70, 384, 144, 6, 2), (400, 272, 256, 3, 2)])
def test_in_8_bits(tokens, hidden, inner, experts, k):
    """A norm's codes gathered with their scales, multiplied, activated into codes
    and multiplied again; and a gradient in codes taken back to the rows."""
    dt = torch.bfloat16
    m = Mlp(tokens, hidden, inner, experts, k, dt, seed=tokens)
    (up, ups), (down, downs) = blocks(m.up), blocks(m.down)
    upd, downd = up.to(DEV), down.to(DEV)
    groups, inner_groups, rows = -(-hidden // 128), -(-inner // 128), m.rows.shape[0]
    codes, scales = m.new(hidden, F8, tokens), m.new(groups, torch.float32, tokens)
    hr.reduce_rmsnorm([m.x], weight=None, out8=codes, scales=scales, group=128)
    hr.experts_sort(m.ids, m.offsets, m.order, m.pos)
    sorted8, sorted_scales = m.new(hidden, F8), m.new(groups, torch.float32)
    hr.experts_gather(codes, m.pos, sorted8, offsets=m.offsets, order=m.order, scales=scales, scales_out=sorted_scales)
    hr.experts_product(sorted8, upd, m.h, offsets=m.offsets, x_scales=sorted_scales, w_scales=ups.to(DEV))
    a8, a_scales = m.new(inner, F8), m.new(inner_groups, torch.float32)
    hr.experts_act(m.h, offsets=m.offsets, out8=a8, scales=a_scales)
    hr.experts_product(a8, downd, m.z, offsets=m.offsets, x_scales=a_scales, w_scales=downs.to(DEV))
    hr.experts_combine(m.z, m.pos, m.y, weights=m.weights)
    # the same on what the codes stand for
    m.x = wide_rows(codes.cpu(), scales.cpu())
    y, _ = m.reference(wide_blocks(up, ups), wide_blocks(down, downs))
    # h and z in bfloat16 (and y), a in e4m3: half a step of 2^-4 of a value, and so of the norm
    assert rel(m.y, y) <= 4 * 2.0 ** -9 + 2.0 ** -4
    dz8, dz_scales = m.new(hidden, F8), m.new(groups, torch.float32)
    dz = torch.randn(rows, hidden, generator=torch.Generator().manual_seed(1)).to(dt).to(DEV)
    hr.experts_act(dz, gated=False, offsets=m.offsets, out8=dz8, scales=dz_scales)
    hr.experts_product(dz8, downd, m.da, offsets=m.offsets, x_scales=dz_scales, w_scales=downs.to(DEV), transposed=True)
    o = m.offsets.tolist()
    ref = torch.cat([dz[a:b].cpu().double() @ wide_blocks(down, downs)[e] for e, (a, b) in enumerate(zip(o, o[1:]))])
    assert rel(m.da[:o[-1]], ref) <= 2.0 ** -9 + 2.0 ** -4
