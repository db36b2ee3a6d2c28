"""The router's training operators against plain 64-bit implementations:
moe_balance_loss (balance and z losses, per-expert counts), moe_route_backward
(the logits' gradient) and moe_combine_backward.

Tolerances count roundings of u = 2^-24 (fp32, half a step relative).  A
probability is 2^(d log2(e)) over the sum of its row's, d = l - max, here >= -20.
Its numerator costs the subtraction (|d| u in the exponent), the product (|d| u,
and 0.22 |d| u for the constant) and the power (2 ulp = 4 u): 49 u.  The
denominator's terms cost the same, each weighed by its p; as sum p |d| <= ln E < 7,
that is 7 * 2.22 u + 4 u < 20 u, and adding them (<= 32 values in a lane, 5 shuffle
steps) 37 u.  With the reciprocal and the product (3 u): 109 u, under P_ERR = 128.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import routed_moe_swiglu_b200 as rm
from moe_testlib import GpuMoe
import workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
P_ERR = 128  # roundings of a probability, see above


def _problem(T, E, k, S, seed, masked=False, cap=None, offsets=None):
    """Inputs on the CPU: logits (NaN past the live rows), ids with probs, dprobs, mask, offsets."""
    g = torch.Generator().manual_seed(seed)
    cap = T if cap is None else cap
    logits = torch.full((cap, E), float("nan"))
    logits[:T] = torch.randn((T, E), generator=g) * 1.5
    ids = torch.full((cap, k), -7, dtype=torch.int32)
    ids[:T] = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int() if T else ids[:0]
    probs = torch.full((cap, k), float("nan"))
    probs[:T] = torch.softmax(torch.randn((T, k), generator=g), dim=1)
    dprobs = torch.full((cap, k), float("nan"))
    dprobs[:T] = torch.randn((T, k), generator=g)
    mask = (torch.rand(cap, generator=g) < 0.7).to(torch.uint8) if masked else None
    if offsets is None and S > 1:
        offsets = [0] + sorted(torch.randint(0, T + 1, (S - 1,), generator=g).tolist()) + [T]
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    return dict(T=T, E=E, k=k, S=S, cap=cap, logits=logits, ids=ids, probs=probs, dprobs=dprobs, mask=mask, off=off)


def _reference(q, coef, zc, grads=(1.0, 1.0), chosen=True):
    """Losses, counts, sums and the gradient in 64 bits, with the size of each
    gradient entry's terms (what its roundings are relative to)."""
    T, E, k, S = q["T"], q["E"], q["k"], q["S"]
    lg = q["logits"][:T].double().numpy()
    off = [0, T] if q["off"] is None else np.clip(q["off"].numpy(), 0, T).tolist()
    top = lg.max(axis=1, initial=-np.inf) if E else None
    alive = top > -np.inf
    if q["mask"] is not None:
        alive &= q["mask"][:T].numpy() != 0
    seq = np.full(T, -1)
    for s in range(S):
        seq[off[s]:off[s + 1]] = s
    alive &= seq >= 0
    lse = np.full(T, -np.inf)
    p = np.zeros((T, E))
    for t in np.nonzero(alive)[0]:
        x = np.exp(lg[t] - top[t])
        lse[t] = top[t] + np.log(x.sum())
        p[t] = x / x.sum()
    counts = np.zeros((S, E), np.int64)
    sums = np.zeros((S, E))
    n = np.zeros(S)
    ids = q["ids"][:T].numpy()
    for t in np.nonzero(alive)[0]:
        n[seq[t]] += 1
        sums[seq[t]] += p[t]
        for e in ids[t]:
            if 0 <= e < E:
                counts[seq[t], e] += 1
    filled, total = int((n > 0).sum()), n.sum()
    a = np.array([coef * E / (filled * k * m * m) if m else 0.0 for m in n])
    z2 = 2 * zc / total if total else 0.0
    losses = np.array([(a * (counts * sums).sum(axis=1)).sum(),
                       zc / total * (lse[alive] ** 2).sum() if total else 0.0])
    d = np.zeros((T, E))
    size = np.zeros((T, E))
    for t in np.nonzero(alive)[0]:
        c = counts[seq[t]]
        dot = (c * p[t]).sum()
        d[t] = p[t] * (grads[0] * a[seq[t]] * (c - dot) + grads[1] * z2 * lse[t])
        size[t] = p[t] * (abs(grads[0]) * a[seq[t]] * (c + dot) + abs(grads[1] * z2) * (abs(lse[t]) + abs(top[t]) + 1))
        if chosen:
            w, g = q["probs"][t].double().numpy(), q["dprobs"][t].double().numpy()
            ok = (ids[t] >= 0) & (ids[t] < E)
            wg, wa = (w * g)[ok].sum(), (w * abs(g))[ok].sum()
            for j in np.nonzero(ok)[0]:
                d[t, ids[t, j]] += w[j] * (g[j] - wg)
                size[t, ids[t, j]] += w[j] * (abs(g[j]) + wa)
    return dict(counts=counts, sums=sums, lse=lse, losses=losses, d=d, size=size, n=n, alive=alive, p=p, a=a, top=top)


class _Run:
    """A plan with the buffers of one problem on the GPU; outputs hold a sentinel."""

    def __init__(self, q):
        f = dict(dtype=torch.float32, device="cuda")
        E, S, cap = q["E"], q["S"], q["cap"]
        self.q = q
        self.plan = rm.moe_plan_create(hidden=64, ffn=64, num_experts=E, top_k=q["k"], capacity=cap)
        self.dev = {n: None if q[n] is None else q[n].cuda() for n in ("logits", "ids", "probs", "dprobs", "mask", "off")}
        self.ws = torch.full((rm.moe_balance_workspace_bytes(self.plan, S),), 0xA5, dtype=torch.uint8, device="cuda")
        self.live = torch.tensor([q["T"]], dtype=torch.int32, device="cuda")
        self.counts = torch.full((S, E), -5, dtype=torch.int32, device="cuda")
        self.sums, self.lse = torch.full((S, E), -5.0, **f), torch.full((cap,), -5.0, **f)
        self.losses, self.scales = torch.full((2,), -5.0, **f), torch.full((S + 1,), -5.0, **f)
        self.dlogits = torch.full((cap, E), -5.0, **f)

    def forward(self, coef, zc, stream=None):
        d = self.dev
        rm.moe_balance_loss(self.plan, d["logits"], d["ids"], self.live, self.counts, self.sums, self.lse, self.losses,
                            self.scales, self.ws, balance_coef=coef, z_coef=zc, token_mask=d["mask"],
                            seq_offsets=d["off"], stream=stream)

    def backward(self, grads=None, chosen=True, losses=True, stream=None):
        d = self.dev
        loss = dict(lse=self.lse, counts=self.counts, grad_scales=self.scales, grad_losses=grads,
                    seq_offsets=d["off"]) if losses else {}
        pick = dict(probs=d["probs"], dprobs=d["dprobs"]) if chosen else {}
        rm.moe_route_backward(self.plan, d["logits"], d["ids"], self.live, self.dlogits, stream=stream, **loss, **pick)


def _check(r, ref, coef, zc, chosen=True):
    q, T, E = r.q, r.q["T"], r.q["E"]
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    sums = r.sums.cpu().double().numpy()
    # a sum of positive terms: P_ERR for each, and at most one rounding for each of its <= T terms' partial sums
    terms = min(max(int(ref["n"].max(initial=0)), 1), 512)
    assert (np.abs(sums - ref["sums"]) <= (P_ERR + terms) * U * ref["sums"]).all()
    lse = r.lse.cpu().double().numpy()
    assert (lse[T:] == -5.0).all(), "rows past the live count were written"
    lse = lse[:T]
    assert np.array_equal(np.isneginf(lse), ~ref["alive"])
    al = ref["alive"]
    lse_err = U * (2 * np.abs(ref["lse"][al]) + 2 * np.abs(ref["top"][al]) + P_ERR)
    assert (np.abs(lse[al] - ref["lse"][al]) <= lse_err).all()
    got = r.losses.cpu().double().numpy()
    # the balance loss: positive terms, a product and a sum over E more than the sums
    assert abs(got[0] - ref["losses"][0]) <= (P_ERR + terms + 64) * U * ref["losses"][0]
    total = max(int(ref["n"].sum()), 1)
    if not zc:
        assert got[1] == 0
    else:
        z_err = zc / total * (2 * np.abs(ref["lse"][al]) * lse_err + terms * U * ref["lse"][al] ** 2).sum()
        assert abs(got[1] - ref["losses"][1]) <= z_err + 4 * U * abs(ref["losses"][1])
    d = r.dlogits.cpu().double().numpy()
    assert (d[T:] == -5.0).all(), "rows past the live count were written"
    # each entry: P_ERR for p, <= 37 + 16 more in the two inner sums, a few products
    err = np.abs(d[:T] - ref["d"]) - (2 * P_ERR + 64) * U * ref["size"]
    assert (err <= 0).all(), (err.max(), np.unravel_index(err.argmax(), err.shape))
    assert (d[:T][~al] == 0).all()


CASES = [  # T, E, k, S, masked, cap
    (1, 1, 1, 1, False, 1), (1, 8, 2, 1, False, 5), (64, 8, 2, 1, False, 64), (5, 17, 3, 2, True, 9),
    (333, 60, 6, 4, True, 400), (31, 64, 4, 1, True, 31), (700, 128, 8, 1, False, 700), (701, 128, 8, 9, True, 800),
    (259, 200, 16, 3, False, 259), (130, 513, 4, 130, False, 131), (97, 1000, 16, 5, True, 97),
    (40, 1023, 16, 1, False, 40), (40, 1024, 16, 2, True, 64), (0, 16, 2, 3, False, 8)]


@pytest.mark.parametrize("T,E,k,S,masked,cap", CASES)
def test_losses_and_gradient(T, E, k, S, masked, cap):
    q = _problem(T, E, k, S, seed=T * 7 + E, masked=masked, cap=cap)
    coef, zc, grads = 0.01, 0.001, (0.7, -1.3)
    r = _Run(q)
    r.forward(coef, zc)
    r.backward(torch.tensor(grads, device="cuda"))
    _check(r, _reference(q, coef, zc, grads), coef, zc)


def test_losses_alone_and_chosen_alone():
    q = _problem(90, 24, 4, 2, seed=3, masked=True, cap=100)
    r = _Run(q)
    r.forward(0.5, 0.0)
    r.backward(chosen=False)
    _check(r, _reference(q, 0.5, 0.0, chosen=False), 0.5, 0.0)
    # the chosen part alone knows no mask: every live token counts
    free = dict(q, mask=None, off=None, S=1)
    r.backward(losses=False)
    ref = _reference(free, 0.0, 0.0)
    d = r.dlogits.cpu().double().numpy()
    assert (np.abs(d[:90] - ref["d"]) <= 64 * U * ref["size"] + 0).all() and (d[90:] == -5.0).all()


def test_sequences_that_are_empty_or_leave_tokens_out():
    """Offsets that start behind token 0, end before the live count, hold empty
    sequences and (the last two) lie behind the live count."""
    for offsets in ([3, 3, 50, 50, 50, 77, 90], [0, 0, 100, 100], [0, 40, 130, 200], [100, 100, 100], [120, 130, 140]):
        q = _problem(100, 40, 4, len(offsets) - 1, seed=len(offsets), masked=True, cap=110, offsets=offsets)
        r = _Run(q)
        r.forward(0.3, 0.1)
        r.backward()
        _check(r, _reference(q, 0.3, 0.1), 0.3, 0.1)


@pytest.mark.parametrize("T,E,k,offsets", [
    (700, 128, 8, [3, 641]), (700, 128, 8, [690, 700]), (70, 1000, 16, [10, 12]), (70, 1000, 16, [5, 5]),
    (3000, 64, 4, [0, 1, 2, 3, 1500, 1501, 2999]), (513, 1024, 8, [0, 500, 503, 505, 513]),
    (900, 16, 2, list(range(0, 200)) + [500, 900]), (257, 257, 3, [0, 100, 100, 130, 200, 257]),
    (300, 8, 1, [0, 17, 34, 51, 68, 85, 102, 119, 136, 153, 170, 187, 204, 300])])
def test_runs_of_every_kind(T, E, k, offsets):
    """Blocks that meet one sequence, some, or many; long ones cut into segments beside short ones;
    tokens before the first and behind the last."""
    q = _problem(T, E, k, len(offsets) - 1, seed=T + E, masked=True, offsets=offsets)
    r = _Run(q)
    r.forward(0.3, 0.02)
    r.backward()
    _check(r, _reference(q, 0.3, 0.02), 0.3, 0.02)


def test_rows_that_nothing_is_left_of():
    """Masked rows may hold anything; a row of -infinity does not count; -infinity and the type's lowest
    value disable experts; ids outside the experts are dropped; a mask of zeros leaves losses of 0."""
    q = _problem(50, 20, 4, 2, seed=11, masked=True)
    q["mask"][:6] = torch.tensor([0, 0, 1, 1, 1, 1], dtype=torch.uint8)
    q["logits"][0] = float("nan")
    q["logits"][1] = float("inf")
    q["probs"][0] = float("nan")
    q["dprobs"][1] = float("inf")
    q["logits"][2] = float("-inf")
    q["logits"][3, ::2] = float("-inf")
    q["logits"][4, 1:] = torch.finfo(torch.float32).min
    q["ids"][5] = torch.tensor([-1, 20, 3, 2 ** 31 - 1], dtype=torch.int32)
    r = _Run(q)
    r.forward(0.3, 0.1)
    r.backward()
    _check(r, _reference(q, 0.3, 0.1), 0.3, 0.1)
    q["mask"].zero_()
    r = _Run(q)
    r.forward(0.3, 0.1)
    r.backward()
    _check(r, _reference(q, 0.3, 0.1), 0.3, 0.1)
    assert r.losses.tolist() == [0.0, 0.0] and r.scales.tolist() == [0.0, 0.0, 0.0]


def test_rows_near_the_bounds_of_the_type():
    """Rows whose experts are all at the type's lowest value (equal shares), and rows far from zero
    (the differences of their logits are exact, lse is not)."""
    q = _problem(30, 24, 3, 1, seed=13)
    q["logits"][3] = torch.finfo(torch.float32).min
    q["logits"][4] = torch.finfo(torch.float32).min
    q["logits"][4, 7] = torch.finfo(torch.float32).max
    q["logits"][8] = torch.round(q["logits"][8] * 1024) / 1024 + 8192
    q["logits"][9] = torch.round(q["logits"][9] * 1024) / 1024 - 8192
    r = _Run(q)
    r.forward(0.3, 0.0)
    r.backward()
    _check(r, _reference(q, 0.3, 0.0), 0.3, 0.0)


def test_nan_in_a_counted_row_shows():
    for bad in (float("nan"), float("inf")):
        q = _problem(20, 12, 2, 2, seed=5, offsets=[0, 10, 20])
        q["logits"][4, 3] = bad
        r = _Run(q)
        r.forward(0.3, 0.1)
        r.backward(chosen=False)
        torch.cuda.synchronize()
        assert torch.isnan(r.losses).all() and torch.isnan(r.sums[0]).all() and torch.isfinite(r.sums[1]).all()
        d = r.dlogits.cpu()
        assert torch.isnan(d[4]).all() and torch.isfinite(d[:4]).all() and torch.isfinite(d[5:]).all()


def test_an_expert_named_twice_gets_both_parts():
    q = _problem(33, 8, 4, 1, seed=9)
    q["ids"][::2, 2] = q["ids"][::2, 0]
    q["ids"][::4, 3] = q["ids"][::4, 0]
    r = _Run(q)
    r.forward(0.3, 0.1)
    r.backward()
    _check(r, _reference(q, 0.3, 0.1), 0.3, 0.1)


def test_logits_and_gradients_at_odd_addresses():
    """Rows of a multiple of four floats that do not start on 16 bytes."""
    q = _problem(37, 64, 3, 1, seed=21)
    r = _Run(q)
    room = torch.empty(37 * 64 + 1, device="cuda")
    room[1:] = r.dev["logits"].reshape(-1)
    r.dev["logits"] = room[1:].view(37, 64)
    r.dlogits = torch.full((37 * 64 + 3,), -5.0, device="cuda")[3:].view(37, 64)
    r.forward(0.2, 0.3)
    r.backward()
    _check(r, _reference(q, 0.2, 0.3), 0.2, 0.3)


def test_gradient_against_differences():
    """The gradient along random directions against central differences of the 64-bit losses (counts
    and routes held) plus the chosen probabilities' sum with dprobs."""
    q = _problem(60, 16, 3, 2, seed=31, masked=True)
    coef, zc, grads = 0.8, 0.05, (1.5, 0.5)
    lg = q["logits"].double()
    ids = q["ids"].long()
    q["probs"] = torch.softmax(lg.gather(1, ids), dim=1).float()
    r = _Run(q)
    r.forward(coef, zc)
    r.backward(torch.tensor(grads, device="cuda"))
    d = r.dlogits.cpu().double()

    def total(x):
        ref = _reference(dict(q, logits=x), coef, zc)
        alive = torch.from_numpy(ref["alive"])
        w = torch.softmax(x.gather(1, ids), dim=1)
        return grads[0] * ref["losses"][0] + grads[1] * ref["losses"][1] + float((w * q["dprobs"].double())[alive].sum())

    g = torch.Generator().manual_seed(1)
    for _ in range(4):
        v = torch.randn(lg.shape, generator=g, dtype=torch.float64)
        h = 1e-4
        num = (total(lg + h * v) - total(lg - h * v)) / (2 * h)
        # third derivatives are O(1) sums of 60 tokens: h^2 * 60 ~ 6e-7; fp32 inputs and roundings: sum |d v| * 1e-5
        assert abs(num - float((d * v).sum())) <= 1e-5 * float((d * v).abs().sum()) + 1e-5


def test_same_bits_every_run_and_in_a_graph():
    """Repeated calls, a captured call replayed with new inputs and a new live count, and a workspace
    with other contents give the bits of a fresh call."""
    q = _problem(901, 96, 6, 7, seed=41, masked=True, cap=1000)
    a, b = _Run(q), _Run(q)
    b.ws.fill_(0xFF)
    for r in (a, b):
        r.forward(0.01, 0.001)
        r.backward()
    torch.cuda.synchronize()
    for n in ("counts", "sums", "lse", "losses", "scales", "dlogits"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.forward(0.01, 0.001)
        b.backward()
    q2 = _problem(640, 96, 6, 7, seed=42, masked=True, cap=1000)
    fresh = _Run(q2)
    fresh.forward(0.01, 0.001)
    fresh.backward()
    for n, t in fresh.dev.items():
        b.dev[n].copy_(t)
    b.live.copy_(fresh.live)
    for n in ("counts", "sums", "lse", "losses", "scales", "dlogits"):
        getattr(b, n).fill_(-5)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for n in ("counts", "sums", "lse", "losses", "scales", "dlogits"):
        assert torch.equal(getattr(fresh, n), getattr(b, n)), n


def test_two_streams_with_a_workspace_each():
    runs = [_Run(_problem(500 + i, 64, 4, 3, seed=50 + i, masked=True)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        for r, s in zip(runs, streams):
            r.forward(0.2, 0.1, stream=s)
            r.backward(stream=s)
    torch.cuda.synchronize()
    for r in runs:
        _check(r, _reference(r.q, 0.2, 0.1), 0.2, 0.1)


def test_many_tokens():
    """More tokens than one pass of the grid holds; sums against torch in 64 bits."""
    T, E, k = 70001, 128, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((T, E), generator=g, device="cuda")
    ids = torch.topk(logits, k, dim=1).indices.int().contiguous()
    q = dict(T=T, E=E, k=k, S=1, cap=T, logits=logits, ids=ids, probs=None, dprobs=None, mask=None, off=None)
    r = _Run(q)
    r.forward(1.0, 0.0)
    p = torch.softmax(logits.double(), dim=1)
    assert torch.equal(r.counts[0].long(), torch.bincount(ids.reshape(-1).long(), minlength=E))
    # a block's <= 473 tokens are added by 64 lane groups, <= 8 each, which meet in 4 + 16 steps; the
    # 148 blocks' sums by 8 warps of <= 19, and these in 8 steps: under 64 roundings
    ref = p.sum(dim=0)
    assert ((r.sums[0].double() - ref).abs() <= (P_ERR + 64) * U * ref).all()
    r.backward(chosen=False)
    c = r.counts[0].double()
    a = E / (k * T * T)
    d = a * p * (c - (p @ c)[:, None])
    size = a * p * (c + (p @ c)[:, None])
    assert ((r.dlogits.double() - d).abs() <= (2 * P_ERR + 64) * U * size).all()


# ---------------------------------------------------------------- the combine's gradient


@pytest.mark.parametrize("T,H,k,out,cap", [
    (1, 8, 1, "fp32", 1), (1, 2048, 16, "bf16", 3), (7, 136, 3, "fp32", 7), (300, 2688, 6, "bf16", 310),
    (33, 4096, 9, "fp32", 40), (5000, 64, 8, "bf16", 5000), (0, 64, 2, "fp32", 4), (70, 512, 16, "bf16", 75),
    (9, 128, 16, "fp32", 9), (45, 248, 13, "fp32", 45), (33, 520, 5, "bf16", 33), (50, 1032, 7, "fp32", 61),
    (3001, 1984, 2, "bf16", 3001), (3, 2056, 16, "fp32", 5), (20011, 80, 1, "fp32", 20011)])
def test_combine_backward(T, H, k, out, cap):
    g = torch.Generator().manual_seed(T + H)
    plan = rm.moe_plan_create(hidden=H, ffn=64, num_experts=16, top_k=k, capacity=cap, out_dtype=out)
    rows = torch.full((cap, k), 2 ** 30, dtype=torch.int32)
    rows[:T] = torch.randperm(T * k + 5, generator=g)[:T * k].view(T, k).int()
    drop = torch.rand((T, k), generator=g) < 0.1
    rows[:T][drop] = -1
    y = torch.randn((T * k + 5, H), generator=g)
    probs = torch.softmax(torch.randn((cap, k), generator=g), dim=1)
    dout = torch.full((cap, H), float("nan"))
    dout[:T] = torch.randn((T, H), generator=g)
    dout = dout.to(torch.bfloat16 if out == "bf16" else torch.float32)
    live = torch.tensor([T], dtype=torch.int32, device="cuda")
    dprobs, dy = torch.full((cap, k), -5.0, device="cuda"), torch.full_like(y, -5.0, device="cuda")
    args = (plan, dout.cuda(), y.cuda(), rows.cuda(), probs.cuda(), live)
    rm.moe_combine_backward(*args, dprobs=dprobs, dy_rows=dy)
    d = dout[:T].double()
    picked = y[rows[:T].long().clamp(min=0)].double()
    ref = torch.where(drop, 0.0, (picked * d[:, None, :]).sum(dim=2))
    size = (picked * d[:, None, :]).abs().sum(dim=2)
    got = dprobs.cpu()
    assert torch.equal(got[T:], torch.full_like(got[T:], -5.0))
    # roundings of a sum: a lane's 4 ceil(H / 4L) products, L = 8 lanes up to H 128, 16 up to 256, 32 up
    # to 2,048 (at most H / 32 + 8), log2 L <= 5 joining them; beyond, 128 threads' H / 128 + 4 and 9
    assert ((got[:T].double() - ref).abs() <= (H / 32 + 16) * U * size).all()
    want = torch.full_like(y, -5.0)
    keep = ~drop
    want[rows[:T][keep].long()] = (probs[:T, :, None] * dout[:T].float()[:, None, :])[keep]
    assert torch.equal(dy.cpu(), want)  # one product each
    only_p, only_y = torch.full_like(dprobs, -5.0), torch.full_like(dy, -5.0)
    rm.moe_combine_backward(*args, dprobs=only_p)
    rm.moe_combine_backward(args[0], args[1], None, *args[3:], dy_rows=only_y)
    assert torch.equal(only_p, dprobs) and torch.equal(only_y, dy)


def test_combine_backward_does_not_depend_on_the_batch():
    """A token's dprobs are the same bits alone (its routes spread over warps) and in a full batch."""
    H, k, T = 1024, 8, 4000
    plan = rm.moe_plan_create(hidden=H, ffn=64, num_experts=16, top_k=k, capacity=T)
    g = torch.Generator(device="cuda").manual_seed(2)
    y, dout = torch.randn((T * k, H), generator=g, device="cuda"), torch.randn((T, H), generator=g, device="cuda")
    rows = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    probs = torch.rand((T, k), generator=g, device="cuda")
    outs = []
    for n in (T, 100, 3):
        d = torch.zeros((T, k), device="cuda")
        rm.moe_combine_backward(plan, dout, y, rows, probs, torch.tensor([n], dtype=torch.int32, device="cuda"), dprobs=d)
        outs.append(d[:3].clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def _view(m, ptr, n, dtype):
    off = ptr - m.ws.data_ptr()
    return m.ws[off:off + 4 * n].view(dtype)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8", "int8"])
def test_a_training_step_of_the_router(precision):
    """Route, losses, experts, then back: the combine's gradient of the forward's own rows into the
    logits' gradient, against the 64-bit chain through the same y rows; and the losses against
    differences of the forward's output along a direction of the logits."""
    H, F, E, k, T, cap = 256, 128, 16, 4, 75, 90
    x, logits, weights = workloads.small_case(H, F, E, k, T, seed=8, capacity=cap)
    m = GpuMoe(H, F, E, k, cap, weights, precision=precision)
    plan, dev = m.plan, "cuda"
    lg = logits.cuda()
    live = torch.tensor([T], dtype=torch.int32, device=dev)
    ids = torch.zeros((cap, k), dtype=torch.int32, device=dev)
    probs = torch.zeros((cap, k), device=dev)
    rm.moe_route_topk(plan, lg, live, ids, probs)
    out = m.forward(x.cuda(), T, logits=lg)
    q = dict(T=T, E=E, k=k, S=1, cap=cap, logits=logits, ids=ids.cpu(), probs=probs.cpu(), dprobs=None, mask=None,
             off=None)
    r = _Run(q)
    r.plan = plan
    r.forward(0.02, 0.003)
    v = m.views()
    y = _view(m, v["y"], v["rows_padded"] * H, torch.float32).view(-1, H)
    inv = _view(m, v["inv"], cap * k, torch.int32).view(cap, k)
    dout = torch.randn((cap, H), generator=torch.Generator(device=dev).manual_seed(4), device=dev)
    dprobs = torch.zeros((cap, k), device=dev)
    rm.moe_combine_backward(plan, dout, y, inv, probs, live, dprobs=dprobs)
    r.dev["dprobs"] = dprobs
    r.backward()
    q["dprobs"] = dprobs.cpu()
    _check(r, _reference(q, 0.02, 0.003), 0.02, 0.003)
    # the chosen part against the output itself: <dout, out(l + h v) - out(l - h v)> / 2h with the
    # experts' rows held (they do not depend on the logits while the choice stays)
    rows = y[inv[:T].long()].double()
    lp = lg[:T].double().gather(1, ids[:T].long())
    w = torch.softmax(lp, dim=1)
    o = (w[:, :, None] * rows).sum(dim=1)
    assert float((o - out[:T].double()).abs().max()) <= 1e-5 * float(rows.abs().max()) * k
    u = torch.randn(lp.shape, dtype=torch.float64, device=dev, generator=torch.Generator(device=dev).manual_seed(5))
    h = 1e-5
    hi, lo = (torch.softmax(lp + s * h * u, dim=1)[:, :, None] * rows for s in (1, -1))
    num = float(((hi - lo).sum(dim=1) * dout[:T].double()).sum()) / (2 * h)
    r.backward(losses=False)
    mine = r.dlogits[:T].double().gather(1, ids[:T].long()) * u
    assert abs(float(mine.sum()) - num) <= 2e-5 * float(mine.abs().sum()) + 1e-6 * float((rows.abs() * dout[:T, None].abs()).sum(2).max())


@pytest.mark.parametrize("grads", [(float("inf"), 1.0), (float("nan"), float("nan")), (-float("inf"), float("inf")), (3e38, 0.0)])
def test_rows_that_do_not_count_stay_zero_when_the_gradient_scale_overflowed(grads):
    """Masked tokens, tokens outside every sequence and rows of -infinity get zeros whatever the losses'
    gradients are, before and behind counted rows that are lost to them."""
    T, E, k = 60000, 60, 4  # several rows after one another in every group of lanes
    q = _problem(T, E, k, 3, seed=31, masked=True, cap=T + 10, offsets=[5, 20000, 20000, 59000])
    q["logits"][40000:40100] = float("-inf")
    alive = q["mask"][:T] != 0
    alive[:5] = alive[59000:] = alive[40000:40100] = False
    r = _Run(q)
    r.forward(1e10, 0.1)
    for chosen in (False, True):
        r.dlogits.fill_(-5.0)
        r.backward(torch.tensor(grads, device="cuda"), chosen=chosen)
        d = r.dlogits.cpu()
        assert not torch.isfinite(d[:T][alive]).all(dim=1).any()
        assert (d[:T][~alive] == 0).all() and (d[T:] == -5.0).all()


@pytest.mark.parametrize("T,E,k,S", [(40, 16, 2, 3), (2000, 64, 4, 200), (3000, 1024, 4, 300), (70000, 32, 2, 90), (5000, 128, 8, 5000)])
def test_offsets_that_decrease(T, E, k, S):
    """Losses and factors are NaN, rows past the live count keep their bytes, and the next call is as ever."""
    good = _problem(T, E, k, S, seed=T, cap=T + 5)
    r = _Run(good)
    r.forward(0.1, 0.1)
    want = [t.clone() for t in (r.losses, r.scales, r.counts, r.sums)]
    assert torch.isfinite(r.losses).all()
    off, g = r.dev["off"], torch.Generator().manual_seed(S)
    tables = [torch.where(torch.arange(S + 1) % 2 == 0, 0, T), torch.randint(-9, T + 9, (S + 1,), generator=g),
              torch.arange(S, -1, -1), torch.cat([off[:-1].cpu(), off[-2:-1].cpu() - 1])]
    if S > 3:  # one decrease in the middle
        tables.append(off.cpu().clone())
        tables[-1][S // 2] = -1 if int(off[S // 2 - 1]) else T
    for table in tables:
        clamped = table.clamp(0, T)
        assert bool((clamped[1:] < clamped[:-1]).any())
        off.copy_(table.int())
        r.forward(0.1, 0.1)
        assert torch.isnan(r.losses).all() and torch.isnan(r.scales).all() and (r.lse[T:] == -5.0).all()
        r.backward()
        assert (r.dlogits[T:] == -5.0).all()
    off.copy_(good["off"])
    r.forward(0.1, 0.1)
    for a, b in zip((r.losses, r.scales, r.counts, r.sums), want):
        assert torch.equal(a, b)
