"""The layer of experts (message_fp16_all_amd/expert_layer.py) against the same
layer in 64 bits with autograd, for the picks that it made; and through host
slots with the same bits."""
import pytest
import torch

from message_fp16_all_amd import expert_layer as el
from message_fp16_all_amd import hr
from _gpu import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


def reference(w, x, ids, dx, dy):
    """(x', y', gradients) in 64 bits on the CPU."""
    leaf = {n: getattr(w, n).detach().cpu().double().requires_grad_() for n in
            ("router", "expert", "scale_in", "scale_out")}
    leaf["x"] = x.cpu().double().requires_grad_()

    def norm(v, scale):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + el.EPS) * scale

    y = norm(leaf["x"], leaf["scale_in"])
    picked = (y @ leaf["router"]).gather(1, ids)
    weights = torch.softmax(picked, 1)
    total = torch.zeros_like(y)
    for e in range(w.expert.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        total = total.index_add(0, t, (y[t] @ leaf["expert"][e]) * weights[t, j, None])
    out = leaf["x"] + total
    y_out = norm(out, leaf["scale_out"])
    ((out * dx.cpu().double()).sum() + (y_out * dy.cpu().double()).sum()).backward()
    return out.detach(), y_out.detach(), {n: v.grad for n, v in leaf.items()}


def rel(got, ref):
    return float((got.detach().cpu().double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,hidden,experts,k,ranks", [(1, 256, 8, 2, 2), (37, 384, 12, 3, 4), (130, 256, 16, 4, 2),
                                                           (33, 200, 6, 6, 1)])
def test_layer(dtype, tokens, hidden, experts, k, ranks):
    w = el.Weights(hidden, experts, dtype, seed=tokens)
    g = torch.Generator().manual_seed(tokens)
    x, dx, dy = (torch.randn(tokens, hidden, generator=g).to(dtype).cuda() for _ in range(3))
    layer = el.Layer(w, tokens, k, ranks)
    print(f"expert layer {tokens} x {hidden}, {experts} experts, k={k}, {ranks} ranks, {dtype}", flush=True)
    x_out, y_out = layer.forward(x)
    grads = layer.backward(dx, dy)
    torch.cuda.synchronize()
    ids = layer.ids.cpu().long()
    assert ((ids >= 0) & (ids < experts)).all()
    xr, yr, gr = reference(w, x, ids, dx, dy)
    half = torch.finfo(dtype).eps / 2
    # 16-bit values on the longest way forward: y, logits, z, a rank's rows, the
    # fold (ranks, the residual), y'; each off by half a step of the larger of
    # what it adds, and the logits' shift every weight
    bound = (8 + ranks) * half
    assert rel(x_out, xr) <= bound and rel(y_out, yr) <= bound
    groups = -(-hidden // 128)
    value = layer.codes.float() * layer.scales.repeat_interleave(128, 1)[:, :hidden]
    assert layer.scales.shape[1] == groups and rel(value, yr) <= bound + 2.0 ** -4
    # the way back has as many again, on values that the way forward rounded
    for name, ref in gr.items():
        assert rel(grads[name], ref) <= 3 * bound, name


def test_through_host_slots_the_same_bits():
    tokens, hidden, ranks = 24, 512, 4
    w = el.Weights(hidden, 16, torch.float16, seed=3)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(2)).half().cuda()
    plain, slots = el.Layer(w, tokens, 4, ranks), el.Layer(w, tokens, 4, ranks, exchange=True)
    try:
        a, b = plain.forward(x), slots.forward(x)
        torch.cuda.synchronize()
        assert slots.channel.status() == hr.HR_OK
        for s, t in zip(a, b):
            assert torch.equal(s.view(torch.int16), t.view(torch.int16))
    finally:
        torch.cuda.synchronize()
        slots.close()


def test_command(capsys):
    el.main(["--tokens", "8", "--hidden", "256", "--experts", "8", "--k", "2", "--bf16"])
    out = capsys.readouterr().out
    assert "forward:" in out and "backward:" in out


def test_as_many_ranks_as_a_fold_takes():
    """Backward then adds a gradient more than one fold takes: every rank's and
    the router's."""
    test_layer(torch.float16, 21, 256, 32, 4, hr.HR_MAX_G)
