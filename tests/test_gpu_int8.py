"""The 8-bit integer operators: int8_quantize_rows, int8_matmul, int8_linear and
the forward of int8 plans, against plain implementations.

The quantiser, the product and every stage of the forward but the SwiGLU are
compared bit for bit: the sums are whole numbers, and the fp32 divisions,
conversions and products that follow round once each, in a stated order.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import routed_moe_swiglu_b200 as rm
import workloads
from moe_testlib import GpuMoe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32, relative


def quantize_ref(x: torch.Tensor):
    """bf16 rows -> (codes int8, scales fp32), in numpy's fp32 (division and rint round as IEEE does)."""
    v = x.float().numpy()
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(axis=-1)
        bad = ~np.isfinite(v).all(axis=-1)
        s = np.where(amax > 0, amax / np.float32(127), np.float32(1)).astype(np.float32)
        s[bad] = np.nan
        q = np.clip(np.rint(v / s[..., None]), -127, 127)
    q[bad] = 0
    return torch.from_numpy(q.astype(np.int8)), torch.from_numpy(s)


def product_ref(xq, xs, wq, ws, bf16):
    """(float(sum) * xs) * ws in fp32, the sum exact (int64), one rounding each."""
    acc = (xq.double() @ wq.double().T).float()  # whole numbers below 2^53: exact, then one rounding
    out = (acc * xs[:, None]) * ws[None, :]
    return out.to(torch.bfloat16) if bf16 else out


def _codes(shape, g, full=True):
    return torch.randint(-128 if full else -127, 128, shape, generator=g, dtype=torch.int16).to(torch.int8)


def _scales(n, g):
    return (torch.rand(n, generator=g) + 0.1) * 0.01


def _same(a, b):
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    both = torch.isnan(a) & torch.isnan(b)
    bad = ~(both | (a == b))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


# ---------------------------------------------------------------- quantiser


@pytest.mark.parametrize("rows,cols,pad", [(1, 8, 0), (3, 16, 8), (17, 104, 0), (5, 2048, 16), (700, 2688, 0), (2, 16384, 0),
                                           (4001, 64, 0)])
def test_quantize_rows(rows, cols, pad):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn((rows, cols + pad), generator=g) * torch.exp(4 * torch.randn((rows, 1), generator=g))
    x = x.to(torch.bfloat16)
    q = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -1.0, device="cuda")
    rm.int8_quantize_rows(x.cuda()[:, :cols], q, s)
    rq, rs = quantize_ref(x[:, :cols])
    _same(s, rs)
    _same(q, rq)


def test_quantize_every_bf16_value():
    """Every finite bf16 as an element of a row whose largest magnitude is each of a few values; rows
    of zeros, of subnormals, with halves (largest / 2), with NaN and infinities."""
    bits = torch.arange(0x8000, dtype=torch.int32)
    every = bits[bits < 0x7F80].to(torch.int16).view(torch.bfloat16)  # 32640 values, ascending
    rows = []
    for top in (1e-38, 1e-30, 0.007, 1.0, 1.9921875, 127.0, 3e5, 3e38):
        v = every.clone()
        v[v.float() > top] = 0
        v[::2] *= -1
        rows.append(v)
    rows += [torch.zeros_like(every), -torch.zeros_like(every), torch.full_like(every, 9.2e-41)]
    for bad in (float("nan"), float("inf"), float("-inf")):
        v = every.clone()
        v[5] = bad
        rows.append(v)
    x = torch.stack(rows)
    assert x.shape[1] % 8 == 0
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(x.shape[0], device="cuda")
    rm.int8_quantize_rows(x.cuda(), q, s)
    rq, rs = quantize_ref(x)
    _same(s, rs)
    _same(q, rq)
    assert torch.isnan(s[-3:]).all() and (q[-3:] == 0).all() and (s[8:10] == 1).all()


@pytest.mark.parametrize("live", [0, 1, 5, 9, -3, 100])
def test_quantize_live_rows(live):
    x = torch.randn((9, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[max(0, min(live, 9)):] = float("nan")
    q = torch.full((9, 64), 99, dtype=torch.int8, device="cuda")
    s = torch.full((9,), -1.0, device="cuda")
    rm.int8_quantize_rows(x.cuda(), q, s, live_rows=torch.tensor([live], dtype=torch.int32, device="cuda"))
    n = max(0, min(live, 9))
    rq, rs = quantize_ref(x[:n]) if n else (x[:0].to(torch.int8), torch.empty(0))
    _same(q[:n], rq)
    _same(s[:n], rs)
    assert (q[n:] == 99).all() and (s[n:] == -1.0).all()


# ---------------------------------------------------------------- product

SHAPES = [(1, 16, 1), (1, 64, 3), (2, 128, 17), (7, 144, 96), (31, 272, 64), (33, 256, 257), (64, 2048, 300),
          (100, 96, 1000), (129, 400, 129), (256, 512, 256), (257, 528, 600), (300, 4096, 512), (600, 1024, 1025),
          (1, 2048, 4096), (16, 8192, 640), (40, 1040, 2000), (5, 16384, 130), (777, 1040, 3712), (600, 2064, 4096),
          (1236, 528, 7678), (1922, 80, 1730)]


@pytest.mark.parametrize("rows,K,N", SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
def test_matmul(rows, K, N, bf16):
    g = torch.Generator().manual_seed(rows * 3 + K + N)
    xq, wq = _codes((rows, K), g), _codes((N, K), g)
    xs, ws = _scales(rows, g), _scales(N, g)
    out = torch.full((rows, N), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rm.int8_matmul(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out, status=status)
    _same(out, product_ref(xq, xs, wq, ws, bf16))
    assert int(status) == 0


def test_largest_sums():
    """The largest K with every product at its largest: the sum stays below 2^31."""
    K = rm.MOE_INT8_MAX_K
    xq = torch.full((3, K), -128, dtype=torch.int8)
    xq[1] = 127
    xq[2, ::2] = 127
    wq = torch.full((2, K), -128, dtype=torch.int8)
    wq[1] = 127
    one = torch.ones(3)
    out = torch.empty((3, 2), device="cuda")
    rm.int8_matmul(xq.cuda(), one.cuda(), wq.cuda(), one[:2].cuda(), out)
    _same(out, product_ref(xq, one, wq, one[:2], False))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,live", [(70, 0), (70, 1), (70, 33), (70, 70), (70, 500), (70, -1), (600, 299), (1500, 1111)])
def test_live_rows_strides_and_odd_addresses(rows, live, bf16):
    """Rows past the live count and columns past N keep their bytes; x rows of a longer stride, out
    rows of an odd stride at an odd address."""
    g = torch.Generator().manual_seed(rows + live)
    K, N = 208, 203
    n = max(0, min(live, rows))
    xq, wq = _codes((rows, K + 48), g), _codes((N, K), g)
    xs, ws = _scales(rows, g), _scales(N, g)
    xs[n:] = float("nan")
    dt = torch.bfloat16 if bf16 else torch.float32
    room = torch.full((rows * 211 + 1,), -5.0, dtype=dt, device="cuda")
    full = room[1:].view(rows, 211)
    rm.int8_matmul(xq.cuda()[:, 16:16 + K], xs.cuda(), wq.cuda(), ws.cuda(), full[:, 3:3 + N],
                   live_rows=torch.tensor([live], dtype=torch.int32, device="cuda"))
    want = torch.full((rows, 211), -5.0, dtype=dt)
    want[:n, 3:3 + N] = product_ref(xq[:n, 16:16 + K], xs[:n], wq, ws, bf16)
    _same(full, want)


def test_out_beyond_two_to_the_31():
    """More than 2^31 output elements: rows at both ends and around the border."""
    rows, K, N = 70000, 16, 40000
    g = torch.Generator().manual_seed(5)
    xq, wq = _codes((rows, K), g), _codes((N, K), g)
    xs, ws = _scales(rows, g), _scales(N, g)
    out = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    rm.int8_matmul(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out)
    border = (1 << 31) // N
    pick = torch.tensor([0, 1, border - 1, border, border + 1, rows - 257, rows - 1])
    _same(out[pick.cuda()], product_ref(xq[pick], xs[pick], wq, ws, True))


def test_rows_do_not_depend_on_the_batch():
    g = torch.Generator().manual_seed(6)
    K, N = 1024, 700
    xq, wq = _codes((600, K), g).cuda(), _codes((N, K), g).cuda()
    xs, ws = _scales(600, g).cuda(), _scales(N, g).cuda()
    whole = torch.empty((600, N), device="cuda")
    rm.int8_matmul(xq, xs, wq, ws, whole)
    for n in (1, 8, 40, 128, 300):
        part = torch.empty((n, N), device="cuda")
        rm.int8_matmul(xq[:n], xs[:n], wq, ws, part)
        _same(part, whole[:n])


@pytest.mark.parametrize("rows,K,N,pad", [(1, 64, 40, 0), (1, 16, 1, 0), (1, 2048, 512, 0), (1, 8192, 4096, 0), (1, 2688, 40000, 0),
                                          (5, 144, 100, 8), (16, 16384, 256, 0), (16, 4112, 333, 16), (13, 2048, 8192, 0),
                                          (17, 2048, 128, 0), (1, 32768, 64, 0), (4, 32768, 40000, 0),
                                          (300, 1040, 777, 24), (33, 4096, 96, 0), (64, 1024, 8000, 0), (65, 1024, 8000, 0)])
def test_linear_is_the_two_calls(rows, K, N, pad):
    g = torch.Generator().manual_seed(rows + K)
    x = torch.randn((rows, K + pad), generator=g).to(torch.bfloat16)
    if rows > 3:
        x[2, 7] = float("nan")
        x[3] = 0
    wq, ws = _codes((N, K), g, full=False), _scales(N, g)
    out = torch.empty((rows, N), device="cuda")
    ws_buf = torch.full((rm.int8_linear_workspace_bytes(rows, K),), 0xEE, dtype=torch.uint8, device="cuda")
    rm.int8_linear(x.cuda()[:, :K], wq.cuda(), ws.cuda(), out, ws_buf)
    q, s = quantize_ref(x[:, :K])
    _same(out, product_ref(q, s, wq, ws, False))
    if rows > 3:
        assert torch.isnan(out[2]).all() and (out[3] == 0).all()


def test_linear_in_a_graph_with_live_counts():
    """One capture serves every live count, and inputs and weights changed between replays are seen."""
    g = torch.Generator().manual_seed(9)
    rows, K, N = 300, 512, 384
    x, live = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    wq, ws = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda")
    out = torch.zeros((rows, N), device="cuda")
    buf = torch.empty(rm.int8_linear_workspace_bytes(rows, K), dtype=torch.uint8, device="cuda")
    rm.int8_linear(x, wq, ws, out, buf, live_rows=live)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rm.int8_linear(x, wq, ws, out, buf, live_rows=live)
    for n in (300, 1, 64, 0, 129):
        xc = torch.randn((rows, K), generator=g).to(torch.bfloat16)
        wc, sc = _codes((N, K), g), _scales(N, g)
        x.copy_(xc), wq.copy_(wc), ws.copy_(sc), live.fill_(n), out.fill_(-5.0)
        graph.replay()
        want = torch.full((rows, N), -5.0)
        q, s = quantize_ref(xc)
        want[:n] = product_ref(q[:n], s[:n], wc, sc, False)
        _same(out, want)


@pytest.mark.parametrize("live", [0, 1, 3, 16, 40, -2])
def test_few_tokens_with_a_live_count(live):
    """Buffers of 16 rows (quantised in the product's launch) and of 40, rows past the live count untouched."""
    g = torch.Generator().manual_seed(14)
    for rows, K, N in ((16, 1040, 200), (40, 1040, 200)):
        n = max(0, min(live, rows))
        x = torch.randn((rows, K), generator=g).to(torch.bfloat16)
        x[n:] = float("nan")
        wq, ws = _codes((N, K), g), _scales(N, g)
        out = torch.full((rows, N + 1), -5.0, device="cuda")
        buf = torch.empty(rm.int8_linear_workspace_bytes(rows, K), dtype=torch.uint8, device="cuda")
        rm.int8_linear(x.cuda(), wq.cuda(), ws.cuda(), out[:, :N], buf,
                       live_rows=torch.tensor([live], dtype=torch.int32, device="cuda"))
        want = torch.full((rows, N + 1), -5.0)
        if n:
            want[:n, :N] = product_ref(*quantize_ref(x[:n]), wq, ws, False)
        _same(out, want)


def test_weights_written_just_before():
    """The product of weights that the call before it has just quantised (no wait between)."""
    g = torch.Generator().manual_seed(10)
    K, N = 2048, 512
    x = torch.randn((4, K), generator=g).to(torch.bfloat16)
    out = torch.empty((4, N), device="cuda")
    buf = torch.empty(rm.int8_linear_workspace_bytes(4, K), dtype=torch.uint8, device="cuda")
    wq, ws = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda")
    xd = x.cuda()
    for i in range(5):
        w = torch.randn((N, K), generator=g).to(torch.bfloat16)
        wd = w.cuda()
        rm.int8_quantize_rows(wd, wq, ws)
        rm.int8_linear(xd, wq, ws, out, buf)
        _same(out, product_ref(*quantize_ref(x), *quantize_ref(w), False))


@pytest.mark.parametrize("rows,K,N", [(17, 2048, 512), (17, 8192, 4096), (100, 4096, 8192), (300, 2048, 512), (700, 2048, 8192)])
def test_weights_written_just_before_larger_products(rows, K, N):
    """The same where the product asks for its weights before its rows are quantised: codes of few tokens
    and wide tiles."""
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn((rows, K), generator=g, device="cuda").to(torch.bfloat16)
    buf = torch.empty(rm.int8_linear_workspace_bytes(rows, K), dtype=torch.uint8, device="cuda")
    ws = [torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    want = []
    for w in ws:  # each with codes of its own and a wait between
        wq, s, out = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda"), torch.zeros((rows, N), device="cuda")
        rm.int8_quantize_rows(w, wq, s)
        torch.cuda.synchronize()
        rm.int8_linear(x, wq, s, out, buf)
        torch.cuda.synchronize()
        want.append(out)
    wq, s = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda")
    outs = [torch.zeros((rows, N), device="cuda") for _ in range(12)]
    for i, out in enumerate(outs):
        rm.int8_quantize_rows(ws[i % 4], wq, s)
        rm.int8_linear(x, wq, s, out, buf)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 4]), i
    pick = torch.arange(0, rows, 16)
    xc, wc = x[pick.cuda()].cpu(), ws[0][:256].cpu()
    _same(want[0][pick.cuda(), :256], product_ref(*quantize_ref(xc), *quantize_ref(wc), False))


def test_no_rows():
    x, w, ws = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(32, 64, dtype=torch.int8, device="cuda"), \
        torch.ones(32, device="cuda")
    q, s, out = torch.zeros(0, 64, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda"), torch.zeros(0, 32, device="cuda")
    buf = torch.zeros(rm.int8_linear_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    rm.int8_quantize_rows(x, q, s)
    rm.int8_matmul(q, s, w, ws, out)
    rm.int8_linear(x, w, ws, out, buf)
    rm.int8_linear(x[:0], w, ws, out, buf)
    torch.cuda.synchronize()


def test_two_streams():
    g = torch.Generator().manual_seed(12)
    jobs = []
    for rows, K, N in ((64, 1024, 512), (500, 768, 640)):
        x = torch.randn((rows, K), generator=g).to(torch.bfloat16)
        wq, ws = _codes((N, K), g), _scales(N, g)
        jobs.append(dict(s=torch.cuda.Stream(), x=x.cuda(), wq=wq.cuda(), ws=ws.cuda(),
                         out=torch.empty((rows, N), device="cuda"),
                         buf=torch.empty(rm.int8_linear_workspace_bytes(rows, K), dtype=torch.uint8, device="cuda"),
                         want=product_ref(*quantize_ref(x), wq, ws, False)))
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            rm.int8_linear(j["x"], j["wq"], j["ws"], j["out"], j["buf"], stream=j["s"])
    torch.cuda.synchronize()
    for j in jobs:
        _same(j["out"], j["want"])


# ---------------------------------------------------------------- the forward


def _pad128(n):
    return (n + 127) // 128 * 128


def _ws(m, ptr, n, dtype):
    off = ptr - m.ws.data_ptr()
    return m.ws[off:off + n * torch.empty((), dtype=dtype).element_size()].view(dtype)


def _check_forward(m, x, weights, ids, probs, out, live, *, relu2=False, clamp=0.0, in_fc1=False, tokens=None):
    """Every stage of the forward from the one before it: x codes and scales, h (bf16) from the exact
    pre-activations, h codes and scales from that h, y from those codes, out from that y."""
    H, F, k = m.H, m.F, m.k
    v = m.views()
    R, hp, fp = v["rows_padded"], _pad128(H), _pad128(F)
    toks = np.arange(live) if tokens is None else tokens
    ids, probs = ids[toks], torch.from_numpy(probs[toks])
    inv = m.read_i32(v["inv"], live * k).reshape(live, k)[toks]
    rows = torch.from_numpy(inv.reshape(-1).astype(np.int64)).cuda()
    tok = torch.from_numpy(np.repeat(toks, k))
    # x
    xq = _ws(m, v["xq"], R * hp, torch.int8).view(R, hp)[rows].cpu()
    xs = _ws(m, v["xq_row_scales"], R, torch.float32)[rows].cpu()
    rq, rs = quantize_ref(x[tok])
    _same(xq[:, :H], rq)
    _same(xs, rs)
    assert (xq[:, H:] == 0).all()
    # h: exact sums, SwiGLU in 64 bits, one bf16 rounding; the kernel's pre-activations carry 3
    # roundings, its exponential and quotient a few more (2 ulp each, the exponent's own rounding
    # |g| u): far inside 2^-16 of the value for |g| <= 80
    e = torch.from_numpy(ids.reshape(-1).astype(np.int64))
    hb = _ws(m, v["h_bf16"], R * fp, torch.bfloat16).view(R, fp)[rows].cpu()
    wq = {n: quantize_ref(w) for n, w in zip(("g", "u", "d"), weights) if w is not None}
    g = torch.empty((len(e), F), dtype=torch.float64)
    u = torch.empty((len(e), F), dtype=torch.float64)
    for ex in e.unique():
        at = e == ex
        for n, dst in (("g", g), ("u", u)):
            if n in wq:
                dst[at] = (rq[at].double() @ wq[n][0][ex].double().T) * rs[at].double()[:, None] * wq[n][1][ex].double()
    if clamp:
        g, u = g.clamp(-clamp, clamp), u.clamp(-clamp, clamp)
    ref = torch.relu(g) ** 2 if relu2 else g / (1 + torch.exp(-g)) * u
    if in_fc1:
        ref = ref * probs.reshape(-1, 1).double()
    # at the clamp's edge and next to zero of relu the values move with their argument
    err = (hb[:, :F].double() - ref).abs() - (2.0 ** -8 + 2.0 ** -16) * ref.abs()
    assert float(err.max()) <= 1e-12, float(err.max())
    assert (hb[:, F:] == 0).all()
    # h codes from the kernel's own h
    hq = _ws(m, v["h"], R * fp, torch.int8).view(R, fp)[rows].cpu()
    hs = _ws(m, v["h_row_scales"], R, torch.float32)[rows].cpu()
    oq, os_ = quantize_ref(hb[:, :F])
    _same(hq[:, :F], oq)
    _same(hs, os_)
    assert (hq[:, F:] == 0).all()
    # y from those codes
    y = _ws(m, v["y"], R * H, torch.float32).view(R, H)[rows].cpu()
    for ex in e.unique():
        at = e == ex
        _same(y[at], product_ref(oq[at], os_[at], wq["d"][0][ex], wq["d"][1][ex], False))
    # out: k fused multiply-adds, one rounding each
    y = y.view(len(toks), k, H).double()
    w = torch.ones_like(probs).double() if in_fc1 else probs.double()
    want = (w[:, :, None] * y).sum(dim=1)
    size = (w[:, :, None] * y).abs().sum(dim=1)
    o = out[torch.from_numpy(toks).cuda()].cpu().double()
    tol = k * U * size + (2.0 ** -8 * want.abs() if m.plan.out_dtype == "bf16" else 0)
    assert ((o - want).abs() <= tol).all()


def _case(H, F, E, k, T, seed, cap=None, zipf=False, **variant):
    x, logits, weights = workloads.small_case(H, F, E, k, T, seed=seed, capacity=cap or T + 16, zipf=zipf)
    m = GpuMoe(H, F, E, k, cap or T + 16, weights, precision="int8", **variant)
    out = m.forward(x.cuda(), T, logits=logits.cuda())
    ids, probs = oracle.route(logits[:T].numpy(), k)
    if variant.get("squared_relu"):
        weights = (weights[0], None, weights[2])
    _check_forward(m, x, weights, ids, probs, out, T, relu2=variant.get("squared_relu", False),
                   clamp=variant.get("gate_up_clamp") or 0.0, in_fc1=variant.get("probs_in_fc1", False))
    assert torch.isnan(out[T:]).all() and m.status() == 0
    return m, x, logits, weights, out


@pytest.mark.parametrize("H,F,E,k,T", [(8, 8, 1, 1, 1), (64, 24, 3, 2, 5), (256, 512, 8, 2, 64), (320, 224, 6, 3, 200),
                                       (136, 392, 7, 7, 33), (512, 1024, 16, 4, 300), (2688, 1856, 4, 2, 1)])
def test_forward(H, F, E, k, T):
    _case(H, F, E, k, T, seed=H + F + 1)


@pytest.mark.parametrize("variant", [dict(squared_relu=True), dict(probs_in_fc1=True, gate_up_clamp=0.75),
                                     dict(out_dtype="bf16"), dict(squared_relu=True, probs_in_fc1=True, gate_up_clamp=0.5)])
def test_forward_variants(variant):
    _case(328, 200, 6, 3, 150, seed=77, **variant)


def test_forward_skewed():
    _case(256, 256, 16, 4, 1500, seed=5, zipf=True)


def test_every_tile_width():
    """Caller routes that give experts 0..513 routes: every tile width, tails and several tiles."""
    H, F, E, k = 320, 224, 20, 2
    counts = np.array([1, 31, 32, 33, 63, 64, 65, 95, 97, 0, 128, 129, 159, 191, 224, 255, 256, 257, 513, 0])
    counts[-1] = counts.sum() % 2
    T = int(counts.sum()) // k
    x, _, weights = workloads.small_case(H, F, E, k, T, seed=79)
    gen = np.random.default_rng(79)
    experts = np.repeat(np.arange(E), counts)
    ids = np.stack([experts[:T], experts[T:]], axis=1)
    ids = ids[gen.permutation(T)].astype(np.int32)
    assert np.all(ids[:, 0] != ids[:, 1])
    p = gen.uniform(0.1, 1.0, size=(T, k))
    probs = (p / p.sum(axis=1, keepdims=True)).astype(np.float32)
    m = GpuMoe(H, F, E, k, T, weights, precision="int8")
    out = m.forward(x.cuda(), T, ids=torch.from_numpy(ids).cuda(), probs=torch.from_numpy(probs).cuda())
    order = np.argsort(ids, axis=1)
    _check_forward(m, x, weights, np.take_along_axis(ids, order, axis=1), np.take_along_axis(probs, order, axis=1), out, T)
    assert m.status() == 0


@pytest.mark.parametrize("H,F,E,k,T,variant", [
    (8, 8, 1, 1, 1, {}), (2688, 1856, 16, 6, 1, {}), (2048, 1024, 12, 8, 2, {}), (264, 136, 5, 2, 4, {}),
    (1032, 520, 4, 4, 3, dict(out_dtype="bf16")), (328, 200, 6, 3, 4, dict(squared_relu=True)),
    (328, 200, 6, 3, 2, dict(probs_in_fc1=True, gate_up_clamp=0.75)),
    (136, 392, 7, 7, 4, dict(squared_relu=True, probs_in_fc1=True, gate_up_clamp=0.5)), (16384, 64, 2, 1, 4, {}),
    (64, 16384, 2, 2, 3, {}), (264, 136, 5, 2, 5, {})])
def test_few_tokens_are_bitwise_the_wide_products(H, F, E, k, T, variant):
    """Plans of at most four live rows (x and h quantised inside the products) give the bits of plans of
    many, in h, in y and in the output, at every live count."""
    x, logits, weights = workloads.small_case(H, F, E, k, T, seed=H + F + T, capacity=T + 3)
    few = GpuMoe(H, F, E, k, T + 3, weights, precision="int8", max_live=T, **variant)
    x2, l2 = (torch.cat([t, t.new_full((300, t.shape[1]), float("nan"))]) for t in (x, logits))
    wide = GpuMoe(H, F, E, k, T + 303, weights, precision="int8", **variant)
    want = wide.forward(x2.cuda(), T, logits=l2.cuda())[:T].clone()
    out = few.forward(x.cuda(), T, logits=logits.cuda())
    assert torch.equal(out[:T], want) and torch.isnan(out[T:]).all() and few.status() == 0
    views = few.views(), wide.views()
    rows = [m.read_i32(v["inv"], T * k) for m, v in zip((few, wide), views)]
    for name, n, dt in (("h_bf16", _pad128(F), torch.bfloat16), ("y", H, torch.float32)):
        a, b = (_ws(m, v[name], v["rows_padded"] * n, dt).view(-1, n)[torch.from_numpy(r).long().cuda()]
                for m, v, r in zip((few, wide), views, rows))
        assert torch.equal(a, b), name
    for n in {0, 1, T // 2, T - 1}:
        out = few.forward(x.cuda(), n, logits=logits.cuda())
        assert torch.equal(out[:n], want[:n]) and torch.isnan(out[n:]).all()


def test_few_tokens_in_a_graph_with_bad_routes_and_nan():
    """One capture of a plan of few rows serves every live count; a dropped token's row is zero, a
    token with a NaN has a row of NaN, the others keep their bits."""
    H, F, E, k, cap = 264, 136, 6, 2, 4
    x, _, weights = workloads.small_case(H, F, E, k, cap, seed=23)
    g = torch.Generator().manual_seed(2)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(cap)]).int()
    probs = torch.softmax(torch.randn((cap, k), generator=g), dim=1)
    m = GpuMoe(H, F, E, k, cap, weights, precision="int8")
    xd, idd, pd = x.cuda(), ids.cuda(), probs.cuda()
    good = m.forward(xd, cap, ids=idd, probs=pd).clone()
    out = torch.zeros((cap, H), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rm.moe_forward(m.plan, xd, m.wbuf, m.live, out, m.ws, ids=idd, probs=pd)
    xd[1, 40] = float("inf")
    idd[2, 1] = E
    for n in (4, 1, 0, 3, 2, 9):
        out.fill_(-7.0)
        m.live.fill_(n)
        graph.replay()
        n = min(n, cap)
        keep = [t for t in range(n) if t not in (1, 2)]
        assert torch.equal(out[keep], good[keep]) and (out[n:] == -7.0).all()
        if n > 1:
            assert torch.isnan(out[1]).all()
        if n > 2:
            assert (out[2] == 0).all()


def test_a_token_of_nan_stays_alone():
    """A NaN or an infinity in one token's row makes that token's output NaN (clamped or not) and
    changes no other token."""
    for clamp in (None, 2.0):
        x, logits, weights = workloads.small_case(256, 128, 8, 2, 40, seed=3)
        m = GpuMoe(256, 128, 8, 2, 40, weights, precision="int8", gate_up_clamp=clamp)
        good = m.forward(x.cuda(), 40, logits=logits.cuda()).clone()
        x[7, 100], x[9, 0] = float("nan"), float("inf")
        bad = m.forward(x.cuda(), 40, logits=logits.cuda())
        keep = [t for t in range(40) if t not in (7, 9)]
        assert torch.isnan(bad[[7, 9]]).all() and torch.equal(bad[keep], good[keep])


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("in_fc1", [False, True])
@pytest.mark.parametrize("huge", [False, True])
def test_gate_times_up_beyond_fp32(T, in_fc1, huge):
    """Finite pre-activations whose product passes fp32's range, the gate far below zero: h is
    silu(gate) * up and stays finite, on plans of few rows and of many."""
    H, F, E = 128, 24, 2
    pairs = [[-80.0, 1e37], [-40.0, 2e38], [-2e19, 2e19], [-60.0, -1e37], [-3e20, -3e20], [0.5, 3.0]]
    if huge:
        pairs += [[2.0, 1e37], [-1.0, 3e38]]
    pairs = torch.tensor(pairs, dtype=torch.float64).repeat(F // len(pairs), 1)
    even = torch.ones(E, F, H, dtype=torch.float64)
    wg, wu = ((even * pairs[:, i].view(1, F, 1) / H).to(torch.bfloat16) for i in (0, 1))
    wd = (torch.randn((E, H, F), generator=torch.Generator().manual_seed(8)) * 1e-20).to(torch.bfloat16)
    x = torch.tensor([1.0, 0.5, 0.9375])[torch.arange(T) % 3].view(T, 1).expand(T, H).to(torch.bfloat16).contiguous()
    ids, probs = (torch.arange(T) % E).int().view(T, 1), torch.full((T, 1), 0.75)
    m = GpuMoe(H, F, E, 1, T, (wg, wu, wd), precision="int8", probs_in_fc1=in_fc1)
    out = m.forward(x.cuda(), T, ids=ids.cuda(), probs=probs.cuda())
    assert m.status() == 0
    v = m.views()
    rows = torch.from_numpy(m.read_i32(v["inv"], T)).long().cuda()
    h = _ws(m, v["h_bf16"], v["rows_padded"] * _pad128(F), torch.bfloat16).view(-1, _pad128(F))[rows].cpu()[:, :F]
    (xq, xs), codes = quantize_ref(x), [quantize_ref(w) for w in (wg, wu)]
    g, u = (torch.stack([(xq[t].double() @ wq[t % E].double().T) * xs[t].double() * ws[t % E].double() for t in range(T)])
            for wq, ws in codes)
    assert torch.isfinite(g.float()).all() and torch.isfinite(u.float()).all() and ((g.float() * u.float()).isinf()).any()
    # three roundings of g and the exponent's own move silu(g) by 4 |g| u; u's, the exponential's, the
    # quotient's and the products' by 16 u more; then the bf16 rounding.  Below -87 the sigmoid is 0.
    ref = g / (1 + torch.exp(-g)) * u * (0.75 if in_fc1 else 1.0)
    assert ((h.double() - ref).abs() <= (2.0 ** -8 + (4 * g.abs().clamp(max=100) + 16) * U) * ref.abs()).all()
    # down: of huge rows the sum times the row's scale, up to 8e37 * 127, passes fp32's range before
    # the channel's scale is applied, as the order of the two products has it
    y = _ws(m, v["y"], v["rows_padded"] * H, torch.float32).view(-1, H)[rows].cpu()
    (hq, hs), (dq, ds) = quantize_ref(h), quantize_ref(wd)
    _same(y, torch.cat([product_ref(hq[t:t + 1], hs[t:t + 1], dq[t % E], ds[t % E], False) for t in range(T)]))
    assert not torch.isnan(out).any() and (huge or torch.isfinite(out).all())


def test_batch_invariance_graph_and_noalloc():
    H, F, E, k = 512, 512, 16, 4
    x, logits, weights = workloads.small_case(H, F, E, k, 600, seed=42)
    m = GpuMoe(H, F, E, k, 600, weights, precision="int8")
    xd, ld = x.cuda(), logits.cuda()
    a = m.forward(xd, 600, logits=ld).clone()
    out = torch.zeros((600, H), device="cuda")
    rm.moe_forward_noalloc(m.plan, xd, m.wbuf, m.live, out, logits=ld)
    assert torch.equal(out, a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rm.moe_forward(m.plan, xd, m.wbuf, m.live, out, m.ws, logits=ld)
    for n in (1, 33, 0, 300, 600):
        out.fill_(-7.0)
        m.live.fill_(n)
        g.replay()
        assert torch.equal(out[:n], a[:n]) and (out[n:] == -7.0).all()


def test_weights_rebuilt_in_place():
    H, F, E, k, T = 264, 136, 5, 2, 50
    m, x, logits, _, _ = _case(H, F, E, k, T, seed=4)
    _, _, other = workloads.small_case(H, F, E, k, T, seed=99)
    m.wbuf.fill_(0xFF)
    m.prepare(other)
    out = m.forward(x.cuda(), T, logits=logits.cuda())
    ids, probs = oracle.route(logits[:T].numpy(), k)
    _check_forward(m, x, other, ids, probs, out, T)


@pytest.mark.parametrize("name,count", [("decode", 256), ("prefill", 96)])
def test_forward_of_the_workloads(name, count):
    """The decode and prefill workloads' shapes with int8 experts; a sample of tokens, and how far the
    result is from the bf16 forward's (two quantisations of 1/254 steps: a few percent)."""
    w = workloads.WORKLOADS[name]
    x, logits = workloads.make_activations(w)
    weights = workloads.make_weights(w)
    m = GpuMoe(w.hidden, w.ffn, w.num_experts, w.top_k, w.capacity, weights, precision="int8", max_live=w.max_live)
    out = m.forward(x.cuda(), w.max_live, logits=logits.cuda(), sentinel=-7.0)
    ids, probs = oracle.route(logits[:w.max_live].numpy(), w.top_k)
    toks = workloads.sample_tokens(w.max_live, min(count, 24), w.seed).numpy()
    _check_forward(m, x, weights, ids, probs, out, w.max_live, tokens=toks)
    assert (out[w.max_live:] == -7.0).all() and m.status() == 0
    ref = oracle.forward_bf16(x[:w.max_live], ids, probs, *weights, tokens=toks)
    d = np.linalg.norm(out.cpu().numpy()[toks] - ref) / np.linalg.norm(ref)
    assert 0.002 < d < 0.05, d


def test_expert_parallel_step_is_the_forward():
    """All ranks' steps in turn on one GPU: the int8 plan's expert-parallel step is bitwise its forward."""
    from routed_moe_swiglu_b200 import ep

    H, F, E, k, T = 256, 128, 8, 3, 70
    m, x, logits, weights, out = _case(H, F, E, k, T, seed=15)
    size, cap = 2, T + 16
    n = m.plan.max_live_rows * k
    dev = dict(device="cuda")
    send_x = torch.zeros((n, H), dtype=torch.bfloat16, **dev)
    send_ids, send_probs = torch.zeros(n, dtype=torch.int32, **dev), torch.zeros(n, **dev)
    counts = torch.zeros(size, dtype=torch.int32, **dev)
    rows = torch.zeros((m.plan.max_live_rows, k), dtype=torch.int32, **dev)
    rp = torch.zeros((m.plan.max_live_rows, k), **dev)
    rm.moe_ep_dispatch(m.plan, size, x.cuda(), m.live, send_x, send_ids, send_probs, counts, rows, rp, m.ws,
                       logits=logits.cuda())
    c = counts.tolist()
    y = torch.zeros((n, H), **dev)
    for rank in range(size):
        first, count = ep.expert_range(E, size, rank)
        shard = ep.shard_plan_create(m.plan, size, n)
        assert shard.precision == "int8"
        buf, ws = rm.alloc_weight_buffer(shard), rm.alloc_workspace(shard)
        rm.moe_prepare_weights(shard, *(t[first:first + count].cuda().contiguous() for t in weights), buf)
        at = sum(c[:rank])
        pad = lambda t: torch.cat([t[at:at + c[rank]], torch.zeros((n - c[rank], *t.shape[1:]), dtype=t.dtype, **dev)])  # noqa: E731
        ry = torch.zeros((n, H), **dev)
        rm.moe_forward(shard, pad(send_x), buf, torch.tensor([c[rank]], dtype=torch.int32, **dev), ry, ws,
                       ids=pad(send_ids).view(-1, 1), probs=pad(send_probs).view(-1, 1))
        y[at:at + c[rank]] = ry[:c[rank]]
    got = torch.full((cap, H), float("nan"), **dev)
    rm.moe_ep_combine(m.plan, y, rows, rp, m.live, got)
    assert torch.equal(got[:T], out[:T])
