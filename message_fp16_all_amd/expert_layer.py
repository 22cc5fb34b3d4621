"""One layer of experts between two all-reduces, forward and backward: how the
operators around the combine are used together.

The experts are spread over the ranks of a group; every rank holds the router,
the norms and the whole batch.  Here all ranks live in one process on one GPU
(as in the loopback exchange).  Forward, with residual stream x (tokens x
hidden, 16 bits):

    y = norm(x)                                         reduce_rmsnorm
    logits = y @ router; weights, ids = top k           router_topk
    per rank: the picks of its experts, sorted          experts_sort
              rows gathered into that order             experts_gather
              every row times its expert's matrix       experts_product
              rows back, weighted and added per token   experts_combine
    x' = x + sum of the ranks' rows; y' = norm(x')      reduce_rmsnorm

The last line folds the ranks' contributions in HBM; with ``exchange`` they go
through host slots (``Channel.allreduce_group``) first and one sum is left to
fold, with the same bits.  ``codes`` also gives y' in e4m3 with a scale per
128 values, as an 8-bit product reads it.

Backward takes the gradients of y' and x' back to those of x and of every
weight.

Usage:  python -m message_fp16_all_amd.expert_layer [--tokens N] [--hidden N]
        [--experts N] [--k N] [--ranks N] [--bf16] [--exchange]
"""
from __future__ import annotations

import argparse

from . import hr

EPS = 1e-6
PAD = 16          # rows that a product's tile wants an expert's segment rounded to


class Weights:
    """The layer's weights on the GPU: ``router`` (hidden x experts), ``expert``
    (one hidden x hidden matrix each) and the norms' ``scale_in``, ``scale_out``."""

    def __init__(self, hidden: int, experts: int, dtype, seed: int = 0):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.router = (torch.randn(hidden, experts, generator=g) / hidden ** 0.5).to(dtype).cuda()
        self.expert = (torch.randn(experts, hidden, hidden, generator=g) / hidden ** 0.5).to(dtype).cuda()
        self.scale_in = (1 + 0.1 * torch.randn(hidden, generator=g)).cuda()
        self.scale_out = (1 + 0.1 * torch.randn(hidden, generator=g)).cuda()


class Layer:
    """The layer for a fixed number of tokens: ``forward`` keeps what
    ``backward`` needs in buffers that are made once."""

    def __init__(self, weights: Weights, tokens: int, k: int, ranks: int, exchange: bool = False):
        import torch
        self.w, self.tokens, self.k, self.ranks = weights, tokens, k, ranks
        hidden, experts = weights.router.shape
        self.hidden, self.experts, self.local = hidden, experts, experts // ranks
        if self.local * ranks != experts:
            raise ValueError(f"{experts} experts over {ranks} ranks")
        dt = weights.router.dtype
        self.channel = hr.Channel(world_size=ranks, max_numel=tokens * hidden) if exchange else None

        def rows(n=tokens, width=hidden, dtype=dt):
            return torch.empty(n, width, dtype=dtype, device="cuda")

        f32 = torch.float32
        self.y, self.x_out, self.y_out = rows(), rows(), rows()
        self.codes, self.scales = rows(dtype=torch.float8_e4m3fn), rows(width=-(-hidden // 128), dtype=f32)
        self.rstd_in, self.rstd_out = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.weights, self.ids = rows(width=k, dtype=f32), rows(width=k, dtype=torch.int32)
        self.sorts = [hr.experts_buffers(tokens, k, self.local, PAD) for _ in range(ranks)]
        self.sorted = [rows(s[1].numel()) for s in self.sorts]
        self.z = [rows(s[1].numel()) for s in self.sorts]
        self.parts = [rows() for _ in range(ranks)]
        self.sums = [rows() for _ in range(ranks)] if exchange else None

    def close(self):
        if self.channel is not None:
            self.channel.destroy()

    def experts_of(self, rank: int) -> slice:
        """A rank's experts."""
        return slice(rank * self.local, (rank + 1) * self.local)

    def forward(self, x):
        """(x', y') of the residual stream ``x``; self.codes and self.scales
        hold y' in 8 bits."""
        import torch
        w = self.w
        self.x = x
        hr.reduce_rmsnorm([x], self.y, weight=w.scale_in, eps=EPS, rstd=self.rstd_in)
        self.logits = torch.mm(self.y, w.router).float()
        hr.router_topk(self.logits, self.weights, self.ids, renormalize=True)
        for r, (offsets, order, pos) in enumerate(self.sorts):
            hr.experts_sort(self.ids, offsets, order, pos, first=r * self.local, pad=PAD)
            hr.experts_gather(self.y, pos, self.sorted[r], offsets=offsets, order=order)
            hr.experts_product(self.sorted[r], w.expert[self.experts_of(r)], self.z[r], offsets=offsets,
                               transposed=True)
            hr.experts_combine(self.z[r], pos, self.parts[r], weights=self.weights)
        parts = self.parts
        if self.channel is not None:
            self.channel.allreduce_group(parts, self.sums)
            parts = self.sums[:1]
        hr.reduce_rmsnorm(parts, self.y_out, residual=x, residual_out=self.x_out, weight=w.scale_out, eps=EPS,
                          out8=self.codes, scales=self.scales, group=128, rstd=self.rstd_out)
        return self.x_out, self.y_out

    def backward(self, dx_out, dy_out):
        """The gradients of x and of the weights, given those of x' and y', as
        a dict.  (scale_in, scale_out in binary32, the others in 16 bits.)"""
        import torch
        w, dt = self.w, self.y.dtype
        g = {"scale_out": torch.empty_like(w.scale_out), "scale_in": torch.empty_like(w.scale_in),
             "expert": torch.empty_like(w.expert)}
        dh = torch.empty_like(self.x)
        hr.rmsnorm_grad(dy_out, self.x_out, self.rstd_out, dh, weight=w.scale_out, dresidual=dx_out,
                        dweight=g["scale_out"])
        # every rank's contribution has the gradient of the sum
        dweights, dys = torch.zeros_like(self.weights), []
        for r, (offsets, order, pos) in enumerate(self.sorts):
            dz, ds, mine = torch.empty_like(self.z[r]), torch.empty_like(self.z[r]), torch.empty_like(self.weights)
            hr.experts_combine_grad(dh, self.z[r], pos, self.weights, dz, mine, offsets=offsets, order=order)
            dweights += mine
            mine_w = self.experts_of(r)
            hr.experts_product(dz, w.expert[mine_w], ds, offsets=offsets)
            hr.experts_product_grad(self.sorted[r], dz, g["expert"][mine_w], offsets=offsets)
            dys.append(hr.experts_combine(ds, pos, torch.empty_like(self.y)))
        dlogits = torch.empty_like(self.logits)
        hr.router_topk_grad(dweights, self.weights, self.ids, dlogits, renormalize=True)
        dlogits = dlogits.to(dt)
        g["router"] = torch.mm(self.y.t(), dlogits)
        dys.append(torch.mm(dlogits, w.router.t()))
        # a fold takes so many operands; the one left over follows, in the same order
        dy = hr.reduce(dys[:hr.HR_MAX_G], torch.empty_like(self.y))
        if len(dys) > hr.HR_MAX_G:
            dy = hr.reduce([dy, *dys[hr.HR_MAX_G:]], torch.empty_like(self.y))
        g["x"] = torch.empty_like(self.x)
        hr.rmsnorm_grad(dy, self.x, self.rstd_in, g["x"], weight=w.scale_in, dresidual=dh, dweight=g["scale_in"])
        return g


def main(argv=None):
    import torch
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--k", type=int, default=4)
    p.add_argument("--ranks", type=int, default=2)
    p.add_argument("--bf16", action="store_true")
    p.add_argument("--exchange", action="store_true")
    a = p.parse_args(argv)
    dt = torch.bfloat16 if a.bf16 else torch.float16
    layer = Layer(Weights(a.hidden, a.experts, dt), a.tokens, a.k, a.ranks, a.exchange)
    try:
        g = torch.Generator().manual_seed(1)
        x, dx, dy = (torch.randn(a.tokens, a.hidden, generator=g).to(dt).cuda() for _ in range(3))
        for name, step in (("forward", lambda: layer.forward(x)), ("backward", lambda: layer.backward(dx, dy))):
            for _ in range(3):
                step()
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(10):
                step()
            end.record()
            end.synchronize()
            print(f"{name}: {start.elapsed_time(end) / 10:.3f} ms")
        load = sum((s[0][1:] - s[0][:-1]).sum() for s in layer.sorts)
        print(f"{a.tokens} tokens x {a.k} picks on {int(load)} rows; |y'| {layer.y_out.float().norm():.1f}, "
              f"its 8-bit form {(layer.codes.float() * layer.scales.repeat_interleave(128, 1)[:, :a.hidden]).norm():.1f}")
    finally:
        torch.cuda.synchronize()
        layer.close()


if __name__ == "__main__":
    main()
