"""Refusals of the router's training operators: host checks before any launch, no GPU needed."""
from __future__ import annotations

import ctypes

import pytest
import torch

import routed_moe_swiglu_b200 as rm

F = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)


def _plan(**kw):
    return rm.moe_plan_create(**dict(dict(hidden=256, ffn=512, num_experts=8, top_k=2, capacity=64), **kw))


def test_balance_workspace_sizes():
    p = _plan()
    one = rm.moe_balance_workspace_bytes(p, 1)
    assert one >= 8 * (64 // 16 + 1) * 8
    assert rm.moe_balance_workspace_bytes(p, 100) > one
    assert rm.moe_balance_workspace_bytes(p, 0) == 0 and rm.moe_balance_workspace_bytes(p, rm.MOE_MAX_SEQS + 1) == 0
    assert rm.load_library().moe_balance_workspace_bytes(None, 1) == 0


def test_balance_loss_rejects_bad_arguments():
    p = _plan()
    n = rm.moe_balance_workspace_bytes(p, 3)

    def call(plan=p.handle, logits=F, ids=F, mask=None, off=F, S=3, coef=0.1, z=0.1, live=F, counts=F, sums=F, lse=F,
             losses=F, scales=F, ws=F, nb=n):
        return rm.load_library().moe_balance_loss(plan, logits, ids, mask, off, S, coef, z, live, counts, sums, lse,
                                                  losses, scales, ws, nb, None)

    for kw in (dict(plan=None), dict(logits=None), dict(ids=None), dict(live=None), dict(counts=None), dict(sums=None),
               dict(lse=None), dict(losses=None), dict(scales=None), dict(ws=None), dict(S=0), dict(S=-1),
               dict(off=None), dict(coef=float("nan")), dict(z=float("inf"))):
        assert call(**kw) == 1, kw
    assert call(S=rm.MOE_MAX_SEQS + 1) == 2
    assert call(nb=n - 1) == 4
    assert call(ws=ODD) == 3


def test_route_backward_rejects_bad_arguments():
    p = _plan()

    def call(plan=p.handle, logits=F, ids=F, lse=F, counts=F, scales=F, grads=None, probs=F, dprobs=F, off=None, S=1,
             live=F, d=F):
        return rm.load_library().moe_route_backward(plan, logits, ids, lse, counts, scales, grads, probs, dprobs, off, S,
                                                    live, d, None)

    for kw in (dict(plan=None), dict(live=None), dict(d=None), dict(logits=None), dict(lse=None), dict(scales=None),
               dict(counts=None), dict(probs=None), dict(dprobs=None), dict(ids=None), dict(S=0), dict(S=2),
               dict(counts=None, scales=None, grads=F),
               dict(counts=None, scales=None, probs=None, dprobs=None)):  # neither part
        assert call(**kw) == 1, kw
    assert call(off=F, S=rm.MOE_MAX_SEQS + 1) == 2


def test_combine_backward_rejects_bad_arguments():
    p = _plan()

    def call(plan=p.handle, dout=F, y=F, rows=F, probs=F, live=F, dp=F, dy=F):
        return rm.load_library().moe_combine_backward(plan, dout, y, rows, probs, live, dp, dy, None)

    for kw in (dict(plan=None), dict(dout=None), dict(rows=None), dict(probs=None), dict(live=None), dict(y=None),
               dict(dp=None, dy=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(dout=ODD), dict(y=ODD), dict(dy=ODD)):
        assert call(**kw) == 3, kw


def test_the_binding_refuses_other_types_and_shapes():
    p = _plan()
    f, i = torch.float32, torch.int32
    ok = dict(logits=torch.zeros(64, 8), ids=torch.zeros(64, 2, dtype=i), live_count=torch.zeros(1, dtype=i),
              counts=torch.zeros(1, 8, dtype=i), prob_sums=torch.zeros(1, 8), lse=torch.zeros(64),
              losses=torch.zeros(2), grad_scales=torch.zeros(2), workspace=torch.zeros(16, dtype=torch.uint8))
    for name, bad in (("logits", torch.zeros(64, 8, dtype=torch.bfloat16)), ("logits", torch.zeros(63, 8)),
                      ("logits", torch.zeros(64, 16)[:, ::2]), ("ids", torch.zeros(64, 2, dtype=torch.int64)),
                      ("ids", torch.zeros(64, 3, dtype=i)), ("counts", torch.zeros(1, 8)),
                      ("prob_sums", torch.zeros(2, 8)), ("lse", torch.zeros(63)), ("losses", torch.zeros(1)),
                      ("grad_scales", torch.zeros(1))):
        with pytest.raises(ValueError):
            rm.moe_balance_loss(p, **dict(ok, **{name: bad}), balance_coef=0.1)
    with pytest.raises(ValueError):
        rm.moe_balance_loss(p, **ok, balance_coef=0.1, token_mask=torch.zeros(64))
    with pytest.raises(ValueError):
        rm.moe_balance_loss(p, **ok, balance_coef=0.1)  # tensors of the host
    with pytest.raises(ValueError):
        rm.moe_route_backward(p, ok["logits"], ok["ids"], ok["live_count"], torch.zeros(64, 8),
                              probs=torch.zeros(64, 2, dtype=torch.float64), dprobs=torch.zeros(64, 2))
    with pytest.raises(ValueError):
        rm.moe_combine_backward(p, torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(128, 256), ok["ids"],
                                torch.zeros(64, 2), ok["live_count"], dprobs=torch.zeros(64, 2))
    with pytest.raises(ValueError):
        rm.moe_combine_backward(p, torch.zeros(64, 256), torch.zeros(128, 255), ok["ids"], torch.zeros(64, 2),
                                ok["live_count"], dprobs=torch.zeros(64, 2))
