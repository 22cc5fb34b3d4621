"""hr_router_topk and its gradient refuse bad arguments before any device call
(CPU): the addresses below are never dereferenced."""
import pytest

from message_fp16_all_amd import hr

BASE = 0x7F0000000000
STEP = 1 << 24
X, W, I, G, D = (BASE + i * STEP for i in range(5))


def topk(logits=X, dtype=hr.HR_DTYPE_F16, tokens=100, experts=64, stride=0, k=8, again=0, weights=W, ids=I):
    return hr.hr_router_topk(logits, dtype, tokens, experts, stride, k, again, weights, ids, 0)


def grad(dweights=G, weights=W, ids=I, logits=X, dtype=hr.HR_DTYPE_F32, tokens=100, experts=64, stride=0, k=8, again=0,
         dlogits=D, dstride=0):
    return hr.hr_router_topk_grad(dweights, weights, ids, logits, dtype, tokens, experts, stride, k, again, dlogits,
                                  dstride, 0)


SHARED = [(dict(k=0), hr.HR_ERR_INVALID_ARG), (dict(k=65), hr.HR_ERR_INVALID_ARG),
          (dict(experts=0), hr.HR_ERR_INVALID_ARG), (dict(dtype=hr.HR_DTYPE_OTHER), hr.HR_ERR_INVALID_ARG),
          (dict(dtype=9), hr.HR_ERR_INVALID_ARG), (dict(k=33), hr.HR_ERR_TOO_LARGE),
          (dict(experts=1025), hr.HR_ERR_TOO_LARGE), (dict(tokens=1 << 31), hr.HR_ERR_TOO_LARGE),
          (dict(tokens=0, logits=None, weights=None, ids=None), hr.HR_OK),
          (dict(weights=None), hr.HR_ERR_INVALID_ARG), (dict(ids=None), hr.HR_ERR_INVALID_ARG),
          (dict(logits=None), hr.HR_ERR_INVALID_ARG), (dict(stride=63), hr.HR_ERR_INVALID_ARG),
          (dict(stride=1 << 61), hr.HR_ERR_INVALID_ARG),
          (dict(logits=X + 1), hr.HR_ERR_ALIGNMENT), (dict(weights=W + 2), hr.HR_ERR_ALIGNMENT),
          (dict(ids=I + 2), hr.HR_ERR_ALIGNMENT)]


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(weights=X + 128), hr.HR_ERR_INVALID_ARG), (dict(ids=X), hr.HR_ERR_INVALID_ARG),
    (dict(ids=W + 4), hr.HR_ERR_INVALID_ARG), (dict(dtype=hr.HR_DTYPE_F32, logits=X + 2), hr.HR_ERR_ALIGNMENT)])
def test_topk_refusals(over, status):
    assert topk(**over) == status


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(dweights=None), hr.HR_ERR_INVALID_ARG), (dict(dlogits=None), hr.HR_ERR_INVALID_ARG),
    (dict(dstride=63), hr.HR_ERR_INVALID_ARG), (dict(dlogits=D + 2), hr.HR_ERR_ALIGNMENT),
    (dict(dweights=G + 1), hr.HR_ERR_ALIGNMENT), (dict(dlogits=X + 4), hr.HR_ERR_INVALID_ARG),
    (dict(dlogits=X, dstride=128), hr.HR_ERR_INVALID_ARG), (dict(dlogits=W), hr.HR_ERR_INVALID_ARG),
    (dict(dlogits=I + 4), hr.HR_ERR_INVALID_ARG), (dict(dlogits=G), hr.HR_ERR_INVALID_ARG),
    (dict(again=1, logits=None, dlogits=None), hr.HR_ERR_INVALID_ARG)])
def test_grad_refusals(over, status):
    assert grad(**over) == status


def test_admission_declines_binary32():
    policy = hr.hr_admit_policy(1, 0, 1, 8)
    assert hr.hr_admit(policy, hr.HR_DTYPE_F32, 2, False, 16) == hr.HR_DECLINE_DTYPE
