"""The short way from Python into the operators (the compiled binding): it takes
the calls that the long way takes, with the same results, and leaves to it every
call that is to be refused."""
from __future__ import annotations

import pytest
import torch

import routed_moe_swiglu_b200 as rm

pytestmark = pytest.mark.gpu

T, E, K, H, S = 37, 24, 3, 64, 2


def _state():
    g = torch.Generator(device="cuda").manual_seed(11)
    f, i = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
    plan = rm.moe_plan_create(hidden=H, ffn=64, num_experts=E, top_k=K, capacity=T)
    s = dict(plan=plan, logits=torch.randn(T, E, generator=g, **f), live=torch.tensor([T - 2], **i),
             ids=torch.stack([torch.randperm(E, generator=g, **f)[:K] for _ in range(T)]).int(),
             mask=(torch.rand(T, generator=g, **f) < 0.8).to(torch.uint8), off=torch.tensor([0, 11, T], **i),
             probs=torch.rand(T, K, generator=g, **f), dprobs=torch.randn(T, K, generator=g, **f),
             counts=torch.zeros(S, E, **i), sums=torch.zeros(S, E, **f), lse=torch.zeros(T, **f),
             losses=torch.zeros(2, **f), scales=torch.zeros(S + 1, **f), dlogits=torch.zeros(T, E, **f),
             grads=torch.tensor([0.5, 2.0], **f), ws=torch.zeros(rm.moe_balance_workspace_bytes(plan, S), dtype=torch.uint8, **f),
             dout=torch.randn(T, H, generator=g, **f), y=torch.randn(T * K, H, generator=g, **f),
             rows=torch.randperm(T * K, generator=g, **f).int().view(T, K), dp=torch.zeros(T, K, **f), dy=torch.zeros(T * K, H, **f),
             x=torch.randn(T, H, generator=g, **f).bfloat16(), w=torch.randint(-127, 128, (40, H), generator=g, dtype=torch.int8, **f),
             w_scales=torch.rand(40, generator=g, **f), q=torch.zeros(T, H, dtype=torch.int8, **f), qs=torch.zeros(T, **f),
             out=torch.zeros(T, 40, **f), out16=torch.zeros(T, 48, dtype=torch.bfloat16, **f)[:, :40],
             buf=torch.zeros(rm.int8_linear_workspace_bytes(T, H), dtype=torch.uint8, **f), status=torch.zeros(1, **i))
    return s


def _calls(s, stream=None):
    """Every operator the compiled binding serves, as functions of overridden arguments."""
    def loss(**o):
        v = {**s, **o}
        rm.moe_balance_loss(v["plan"], v["logits"], v["ids"], v["live"], v["counts"], v["sums"], v["lse"], v["losses"],
                            v["scales"], v["ws"], balance_coef=0.3, z_coef=v.get("z", 0.01), token_mask=v["mask"],
                            seq_offsets=v["off"], stream=stream)

    def grad(**o):
        v = {**s, **o}
        rm.moe_route_backward(v["plan"], v["logits"], v["ids"], v["live"], v["dlogits"], lse=v["lse"], counts=v["counts"],
                              grad_scales=v["scales"], grad_losses=v["grads"], probs=v["probs"], dprobs=v["dprobs"],
                              seq_offsets=v["off"], stream=stream)

    def combine(**o):
        v = {**s, **o}
        rm.moe_combine_backward(v["plan"], v["dout"], v["y"], v["rows"], v["probs"], v["live"], dprobs=v["dp"],
                                dy_rows=v["dy"], stream=stream)

    def quantize(**o):
        v = {**s, **o}
        rm.int8_quantize_rows(v["x"], v["q"], v["qs"], live_rows=v["live"], stream=stream)

    def matmul(**o):
        v = {**s, **o}
        rm.int8_matmul(v["q"], v["qs"], v["w"], v["w_scales"], v["out"], live_rows=v["live"], status=v["status"], stream=stream)

    def linear(**o):
        v = {**s, **o}
        rm.int8_linear(v["x"], v["w"], v["w_scales"], v["out16"], v["buf"], live_rows=v["live"], status=v["status"],
                       stream=stream)
    return dict(loss=loss, grad=grad, combine=combine, quantize=quantize, matmul=matmul, linear=linear)


OUTPUTS = ("counts", "sums", "lse", "losses", "scales", "dlogits", "dp", "dy", "q", "qs", "out", "out16")


def _run(stream=None):
    s = _state()
    torch.cuda.synchronize()
    for f in _calls(s, stream).values():
        f()
    torch.cuda.synchronize()
    return s


def _no_long_way(*tensors):
    raise AssertionError("the call went the long way")


@pytest.fixture
def short():
    rm.load_library()
    if rm._short is None:
        pytest.skip("the compiled binding is not built, or this torch has no exchange table")


def test_same_results_as_the_long_way(short, monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(rm, "_ptrs", _no_long_way)
        a = _run()
    with monkeypatch.context() as m:
        m.setattr(rm, "_short", None)
        b = _run()
    for n in OUTPUTS:
        assert torch.equal(a[n], b[n]), n


def test_streams(short, monkeypatch):
    monkeypatch.setattr(rm, "_ptrs", _no_long_way)
    a, other = _run(), torch.cuda.Stream()
    b = _run(other)
    with torch.cuda.stream(other):
        c = _run()
    for n in OUTPUTS:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]), n
    # the current stream is the one captured: nothing would be recorded on another
    s = _state()
    calls = _calls(s)
    for f in calls.values():
        f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for f in calls.values():
            f()
    for n in OUTPUTS:
        s[n].zero_()
    g.replay()
    torch.cuda.synchronize()
    for n in OUTPUTS:
        assert torch.equal(a[n], s[n]), n


def test_parameters_and_leaves(short, monkeypatch):
    monkeypatch.setattr(rm, "_ptrs", _no_long_way)
    s = _state()
    _calls(s)["loss"](logits=torch.nn.Parameter(s["logits"]))
    first = s["losses"].clone()
    _calls(s)["loss"](logits=s["logits"].clone().requires_grad_())
    assert torch.equal(first, s["losses"]) and float(first[0]) > 0


def _views(t):
    """Tensors of t's values that the operators refuse: other strides, types and a host copy."""
    yield t.cpu()
    yield t.double() if t.is_floating_point() else t.to(torch.int16)
    if t.dim() == 2 and t.shape[0] > 1:
        yield t.t().contiguous().t()
        yield t[:-1, :-1]
    if t.dim() == 1 and t.numel() > 1:
        yield t[:-1]
        yield t.repeat(2)[::2]


NAMES = dict(loss=["logits", "ids", "live", "counts", "sums", "lse", "losses", "scales", "mask", "off"],
             grad=["logits", "ids", "live", "dlogits", "lse", "counts", "scales", "grads", "probs", "dprobs", "off"],
             combine=["dout", "y", "rows", "probs", "live", "dp", "dy"], quantize=["x", "q", "qs", "live"],
             matmul=["q", "qs", "w", "w_scales", "out", "live", "status"],
             linear=["x", "w", "w_scales", "out16", "live", "status"])


@pytest.mark.parametrize("op", list(NAMES))
def test_what_the_long_way_refuses_is_refused(op, monkeypatch):
    s = _state()
    f = _calls(s)[op]
    f()
    refused = 0
    for name in NAMES[op]:
        for bad in _views(s[name]):
            with monkeypatch.context() as m:  # what the long way says of it
                m.setattr(rm, "_short", None)
                try:
                    f(**{name: bad})
                    continue  # it takes it (a dense slice of a longer list, say)
                except (ValueError, rm.MoeError) as e:
                    kind = type(e)
            with pytest.raises(kind):
                f(**{name: bad})
            refused += 1
    assert refused >= 2 * len(NAMES[op])
    torch.cuda.synchronize()


def test_a_closed_plan_is_refused():
    s = _state()
    s["plan"].close()
    for op in ("loss", "grad", "combine"):
        with pytest.raises(rm.MoeError):
            _calls(s)[op]()


def test_values_are_checked_as_before():
    s = _state()
    for z in (float("nan"), float("inf"), 1e300):
        with pytest.raises(rm.MoeError):
            _calls(s)["loss"](z=z)
    with pytest.raises(rm.MoeError):
        _calls(s)["loss"](ws=s["ws"][:-256])
    with pytest.raises(rm.MoeError):
        _calls(s)["linear"](buf=s["buf"][:-256])
    with pytest.raises(rm.MoeError):
        _calls(s)["linear"](x=torch.zeros(T * H + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H))
    _calls(s)["loss"](z=1)  # a whole number is a number
    torch.cuda.synchronize()
