"""Cases of the router's training operators and of the 8-bit integer products.

Four operators, each in its plain form (elementary torch operations) and, where
``own`` is true, through this package's entry points:

  route     the router's balance loss and z loss with per-expert counts, and the
            gradient of the logits (the losses' part and the chosen experts'
            renormalised probabilities' part): moe_balance_loss, moe_route_backward
  combine   the gradient of the combine of the expert rows: moe_combine_backward
  linear    x [T, K] bf16 times 8-bit weights [N, K], a scale for each token and for
            each channel, the tokens quantised in the call: int8_linear
  moe       the routed SwiGLU forward with 8-bit experts: moe_forward of an int8 plan
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases


def listed():
    return [
        # the router of a small test model, one short batch: launch latency counts
        {"name": "route_tiny", "op": "route", "tokens": 64, "experts": 8, "top_k": 2, "seqs": 1, "masked": False},
        # a micro-batch of ragged sequences with padding inside, a balance loss for each sequence
        {"name": "route_sequences", "op": "route", "tokens": 4099, "experts": 128, "top_k": 8, "seqs": 7, "masked": True},
        # very many experts, an odd count, sixteen chosen
        {"name": "route_wide", "op": "route", "tokens": 3001, "experts": 1000, "top_k": 16, "seqs": 1, "masked": True},
        # a whole step's tokens as one batch
        {"name": "route_large", "op": "route", "tokens": 65536, "experts": 128, "top_k": 8, "seqs": 16, "masked": False},
        # a short ragged batch, bf16 output gradients
        {"name": "combine_ragged", "op": "combine", "tokens": 333, "hidden": 2688, "top_k": 6, "out": "bf16"},
        # a training micro-batch, fp32 output gradients
        {"name": "combine_large", "op": "combine", "tokens": 8192, "hidden": 2048, "top_k": 8, "out": "fp32"},
        # one decoded token through a dense projection
        {"name": "linear_token", "op": "linear", "tokens": 1, "cols_in": 2048, "cols_out": 4096, "out": "bf16"},
        # a ragged chunk of a prompt, a width that is no multiple of a tile, fp32 out
        {"name": "linear_ragged", "op": "linear", "tokens": 777, "cols_in": 2688, "cols_out": 3712, "out": "fp32"},
        # a large prompt batch through a wide projection
        {"name": "linear_large", "op": "linear", "tokens": 8192, "cols_in": 8192, "cols_out": 8192, "out": "bf16"},
        # one decoded token through the experts of the live-count sweep's model
        {"name": "moe_token", "op": "moe", "tokens": 1, "hidden": 2688, "ffn": 1856, "experts": 128, "top_k": 6,
         "skewed": False},
        # a decode batch: every expert's weights are read for a few rows each
        {"name": "moe_decode", "op": "moe", "tokens": 256, "hidden": 2048, "ffn": 1024, "experts": 128, "top_k": 8,
         "skewed": False},
        # a prompt batch with a skewed router
        {"name": "moe_prefill", "op": "moe", "tokens": 8192, "hidden": 2048, "ffn": 1024, "experts": 128, "top_k": 8,
         "skewed": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "combine", "linear", "moe"])
    if op == "route":
        experts = _spread(rng, 2, 1024)
        tokens = _spread(rng, 1, max(2, min(65536, 65536 * 128 // experts)))
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": min(experts, rng.randint(1, 16)),
                "seqs": min(tokens, _spread(rng, 1, 64)), "masked": rng.random() < 0.5}
    if op == "combine":
        hidden, top_k = 8 * _spread(rng, 8, 512), rng.randint(1, 16)
        return {"op": op, "tokens": _spread(rng, 1, max(2, 8192 * 2048 * 8 // (hidden * top_k))), "hidden": hidden,
                "top_k": top_k, "out": rng.choice(["bf16", "fp32"])}
    if op == "linear":
        cols_in, cols_out = 16 * _spread(rng, 4, 512), _spread(rng, 16, 8192)
        return {"op": op, "tokens": _spread(rng, 1, 8192), "cols_in": cols_in, "cols_out": cols_out,
                "out": rng.choice(["bf16", "fp32"])}
    experts = _spread(rng, 4, 128)
    return {"op": op, "tokens": _spread(rng, 1, 4096), "hidden": 8 * _spread(rng, 16, 256), "ffn": 8 * _spread(rng, 16, 128),
            "experts": experts, "top_k": min(experts, rng.randint(1, 8)), "skewed": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _routes(logits, k):
    """The k largest logits' experts in ascending id (int32) and their renormalised probabilities."""
    ids = torch.sort(torch.topk(logits, k, dim=1).indices, dim=1).values
    return ids.to(torch.int32).contiguous(), torch.softmax(logits.gather(1, ids), dim=1)


def _logits(gen, tokens, experts, skewed):
    logits = _randn(gen, tokens, experts)
    if skewed:  # a popularity that falls with the rank
        logits -= 1.1 * torch.log1p(torch.randperm(experts, generator=gen, device="cuda").float())
    return logits


def prepare(case, seed):
    gen = _generator(seed)
    s = {"case": case}
    if case["op"] == "route":
        _prepare_route(case, gen, s)
    elif case["op"] == "combine":
        _prepare_combine(case, gen, s)
    elif case["op"] == "linear":
        T, K, N = case["tokens"], case["cols_in"], case["cols_out"]
        s["x"] = _randn(gen, T, K).to(torch.bfloat16)
        s["wq"], s["ws"] = _quantize((_randn(gen, N, K) / math.sqrt(K)).to(torch.bfloat16))
        s["out"] = torch.empty((T, N), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device="cuda")
        if own:
            import routed_moe_swiglu_b200 as rm

            s["ws_buf"] = torch.empty(rm.int8_linear_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    else:
        _prepare_moe(case, gen, s)
    return s


def _prepare_route(case, gen, s):
    T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    s["logits"] = _logits(gen, T, E, True)
    s["ids"], s["probs"] = _routes(s["logits"], k)
    s["dprobs"] = _randn(gen, T, k)
    s["mask"] = (torch.rand(T, generator=gen, device="cuda") < 0.9).to(torch.uint8) if case["masked"] else None
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=gen, device="cuda")).values
    edge = torch.tensor([0, T], device="cuda")
    s["offsets"] = torch.cat([edge[:1], cuts, edge[1:]]).to(torch.int32)
    s["grads"] = torch.tensor([1.0, 0.5], device="cuda")
    s["balance"], s["z"] = 1e-2, 1e-3
    if own:
        import routed_moe_swiglu_b200 as rm

        f32 = dict(dtype=torch.float32, device="cuda")
        s["plan"] = rm.moe_plan_create(hidden=128, ffn=128, num_experts=E, top_k=k, capacity=T)
        s["ws_buf"] = torch.empty(rm.moe_balance_workspace_bytes(s["plan"], S), dtype=torch.uint8, device="cuda")
        s["live"] = torch.tensor([T], dtype=torch.int32, device="cuda")
        s["counts"] = torch.empty((S, E), dtype=torch.int32, device="cuda")
        s["prob_sums"], s["lse"] = torch.empty((S, E), **f32), torch.empty(T, **f32)
        s["losses"], s["grad_scales"] = torch.empty(2, **f32), torch.empty(S + 1, **f32)
        s["dlogits"] = torch.empty((T, E), **f32)


def _prepare_combine(case, gen, s):
    T, H, k = case["tokens"], case["hidden"], case["top_k"]
    dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    s["y"] = _randn(gen, T * k, H)
    s["rows"] = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).view(T, k)
    s["probs"] = torch.softmax(_randn(gen, T, k), dim=1)
    s["dout"] = _randn(gen, T, H).to(dtype)
    if own:
        import routed_moe_swiglu_b200 as rm

        s["plan"] = rm.moe_plan_create(hidden=H, ffn=128, num_experts=max(k, 16), top_k=k, capacity=T, out_dtype=case["out"])
        s["live"] = torch.tensor([T], dtype=torch.int32, device="cuda")
        s["dprobs"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        s["dy"] = torch.empty_like(s["y"])


def _prepare_moe(case, gen, s):
    T, H, F, E, k = (case[n] for n in ("tokens", "hidden", "ffn", "experts", "top_k"))
    s["x"] = _randn(gen, T, H).to(torch.bfloat16)
    s["ids"], s["probs"] = _routes(_logits(gen, T, E, case["skewed"]), k)
    # room for the busiest expert's rows in the plain form's padded batches
    s["room"] = int(torch.bincount(s["ids"].reshape(-1).long(), minlength=E).max())
    w1 = torch.empty((E, 2 * F, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.empty((E, H, F), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w1[e] = _randn(gen, 2 * F, H) / math.sqrt(H)
        w2[e] = _randn(gen, H, F) / math.sqrt(F)
    s["w1q"] = torch.empty((E, 2 * F, H), dtype=torch.int8, device="cuda")
    s["w2q"] = torch.empty((E, H, F), dtype=torch.int8, device="cuda")
    s["w1s"], s["w2s"] = torch.empty((E, 2 * F), device="cuda"), torch.empty((E, H), device="cuda")
    for e in range(E):
        s["w1q"][e], s["w1s"][e] = _quantize(w1[e])
        s["w2q"][e], s["w2s"][e] = _quantize(w2[e])
    s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    if own:
        import routed_moe_swiglu_b200 as rm

        s["plan"] = rm.moe_plan_create(hidden=H, ffn=F, num_experts=E, top_k=k, capacity=T, precision="int8",
                                       out_dtype="bf16")
        s["wbuf"] = rm.alloc_weight_buffer(s["plan"])
        rm.moe_prepare_weights(s["plan"], w1[:, :F].contiguous(), w1[:, F:].contiguous(), w2, s["wbuf"])
        s["ws_buf"] = rm.alloc_workspace(s["plan"])
        s["live"] = torch.tensor([T], dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plain forms


def _quantize(x):
    """Rows of x as whole numbers of [-127, 127] (int8) and a scale for each row, amax / 127."""
    x = x.float()
    amax = x.abs().amax(dim=-1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 127.0), torch.ones_like(amax))
    return torch.round(x / scale[..., None]).clamp(-127, 127).to(torch.int8), scale


def _plain_route(s):
    T, E, k, S = (s["case"][n] for n in ("tokens", "experts", "top_k", "seqs"))
    logits, ids = s["logits"], s["ids"].long()
    counted = torch.ones(T, device="cuda") if s["mask"] is None else s["mask"].float()
    seq = torch.searchsorted(s["offsets"][1:].long().contiguous(), torch.arange(T, device="cuda"), right=True)
    top = logits.amax(dim=1, keepdim=True)
    exps = torch.exp(logits - top)
    total = exps.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    p = exps / total * counted[:, None]
    seq_tokens = torch.zeros(S, device="cuda").index_add_(0, seq, counted)
    prob_sums = torch.zeros((S, E), dtype=torch.float64, device="cuda").index_add_(0, seq, p.double()).float()
    hits = torch.zeros((T, E), device="cuda").scatter_(1, ids, 1.0) * counted[:, None]
    counts = torch.zeros((S, E), device="cuda").index_add_(0, seq, hits)
    filled = (seq_tokens > 0).sum()
    weight = torch.where(seq_tokens > 0, s["balance"] * E / (k * filled * seq_tokens.clamp(min=1.0) ** 2), torch.zeros_like(seq_tokens))
    tokens = seq_tokens.sum()
    z_weight = s["z"] / tokens.clamp(min=1.0)
    losses = torch.stack([(weight * (counts * prob_sums).sum(dim=1)).sum(), z_weight * (lse * lse * counted).double().sum().float()])
    pull = counts[seq]
    inner = pull - (pull * p).sum(dim=1, keepdim=True)
    dlogits = p * (s["grads"][0] * weight[seq][:, None] * inner + s["grads"][1] * 2.0 * z_weight * lse[:, None])
    w, g = s["probs"], s["dprobs"]
    chosen = w * (g - (w * g).sum(dim=1, keepdim=True)) * counted[:, None]
    dlogits = dlogits.scatter_add(1, ids, chosen)
    lse = torch.where(counted > 0, lse, torch.full_like(lse, -math.inf))
    return {"counts": counts.to(torch.int32), "prob_sums": prob_sums, "lse": lse, "losses": losses, "dlogits": dlogits}


def _plain_combine(s):
    y = s["y"][s["rows"].long()]
    dout = s["dout"].float()
    dprobs = (y * dout[:, None, :]).sum(dim=2)
    dy = torch.empty_like(s["y"])
    dy[s["rows"].long().reshape(-1)] = (s["probs"][:, :, None] * dout[:, None, :]).reshape(-1, dout.shape[1])
    return {"dprobs": dprobs, "dy": dy}


def _plain_linear(s):
    xq, xs = _quantize(s["x"])
    acc = xq.float() @ s["wq"].float().t()
    return (acc * xs[:, None] * s["ws"][None, :]).to(s["out"].dtype)


def _plain_moe(s):
    T, H, F, E, k = (s["case"][n] for n in ("tokens", "hidden", "ffn", "experts", "top_k"))
    room = s["room"]
    xq, xs = _quantize(s["x"])
    ids = s["ids"].reshape(-1).long()
    order = torch.argsort(ids, stable=True)
    first = torch.searchsorted(ids[order], torch.arange(E, device="cuda"))
    slot = torch.empty_like(ids)
    slot[order] = ids[order] * room + torch.arange(T * k, device="cuda") - first[ids[order]]
    token = torch.arange(T * k, device="cuda") // k
    rows = torch.zeros((E * room, H), device="cuda")
    rows[slot] = xq[token].float()
    scales = torch.zeros(E * room, device="cuda")
    scales[slot] = xs[token]
    pre = torch.bmm(rows.view(E, room, H), s["w1q"].float().transpose(1, 2)) * scales.view(E, room, 1) * s["w1s"][:, None, :]
    gate, up = pre[..., :F], pre[..., F:]
    h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)
    hq, hs = _quantize(h)
    y = torch.bmm(hq.float(), s["w2q"].float().transpose(1, 2)) * hs[..., None] * s["w2s"][:, None, :]
    y = y.view(E * room, H)[slot].view(T, k, H)
    return (s["probs"][:, :, None] * y).sum(dim=1).to(torch.bfloat16)


# ---------------------------------------------------------------- one pass


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"route": _plain_route, "combine": _plain_combine, "linear": _plain_linear, "moe": _plain_moe}[op](s)
    import routed_moe_swiglu_b200 as rm

    if op == "route":
        rm.moe_balance_loss(s["plan"], s["logits"], s["ids"], s["live"], s["counts"], s["prob_sums"], s["lse"], s["losses"],
                            s["grad_scales"], s["ws_buf"], balance_coef=s["balance"], z_coef=s["z"], token_mask=s["mask"],
                            seq_offsets=s["offsets"])
        rm.moe_route_backward(s["plan"], s["logits"], s["ids"], s["live"], s["dlogits"], lse=s["lse"], counts=s["counts"],
                              grad_scales=s["grad_scales"], grad_losses=s["grads"], probs=s["probs"], dprobs=s["dprobs"],
                              seq_offsets=s["offsets"])
        return {"counts": s["counts"], "prob_sums": s["prob_sums"], "lse": s["lse"], "losses": s["losses"],
                "dlogits": s["dlogits"]}
    if op == "combine":
        rm.moe_combine_backward(s["plan"], s["dout"], s["y"], s["rows"], s["probs"], s["live"], dprobs=s["dprobs"],
                                dy_rows=s["dy"])
        return {"dprobs": s["dprobs"], "dy": s["dy"]}
    if op == "linear":
        rm.int8_linear(s["x"], s["wq"], s["ws"], s["out"], s["ws_buf"])
        return s["out"]
    rm.moe_forward(s["plan"], s["x"], s["wbuf"], s["live"], s["out"], s["ws_buf"], ids=s["ids"], probs=s["probs"])
    return s["out"]


def work(case):
    T = case["tokens"]
    if case["op"] == "route":
        E, k, S = case["experts"], case["top_k"], case["seqs"]
        return {"bytes": T * (8 * E + 12 * k + 4) + (T if case["masked"] else 0) + 8 * S * E, "flops": 12 * T * E}
    if case["op"] == "combine":
        H, k = case["hidden"], case["top_k"]
        return {"bytes": T * k * (8 * H + 12) + T * H * (2 if case["out"] == "bf16" else 4), "flops": 3 * T * k * H}
    if case["op"] == "linear":
        K, N = case["cols_in"], case["cols_out"]
        return {"bytes": 2 * T * K + N * K + 4 * N + T * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * N * K}
    H, F, E, k = (case[n] for n in ("hidden", "ffn", "experts", "top_k"))
    return {"bytes": min(E, T * k) * (3 * H * F + 4 * (2 * F + H)) + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * F}


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, s)
    if op == "combine":
        flat, dout = s["rows"].long().reshape(-1), s["dout"].double()
        token = torch.arange(flat.numel(), device="cuda") // case["top_k"]
        dy = torch.empty_like(s["y"], dtype=torch.float64)
        dprobs = torch.empty(flat.numel(), dtype=torch.float64, device="cuda")
        for at in range(0, flat.numel(), 8192):
            r, d = flat[at:at + 8192], dout[token[at:at + 8192]]
            dprobs[at:at + 8192] = torch.einsum("rh,rh->r", s["y"][r].double(), d)
            dy[r] = d * s["probs"].reshape(-1)[at:at + 8192].double()[:, None]
        return {"dprobs": dprobs.view(case["tokens"], case["top_k"]), "dy": dy}
    if op == "linear":
        xq, xs = _exact_codes(s["x"])
        return torch.einsum("tk,nk->tn", xq, s["wq"].double()) * torch.outer(xs, s["ws"].double())
    return _exact_moe(case, s)


def _exact_codes(x):
    """The quantiser's definition: the scale is amax / 127 rounded to fp32 (1 for a row of zeros), the
    codes are the nearest whole numbers of value / scale rounded to fp32, halves to even (a value of half
    the largest is such a half in every row; a quotient of 64 bits rounded to 32 is rounded as if once)."""
    x = x.double()
    biggest = x.abs().max(dim=-1).values
    scale = (biggest / 127).to(torch.float32).double()
    scale[biggest == 0] = 1.0
    quotient = (x / scale.unsqueeze(-1)).to(torch.float32).double()
    return torch.round(quotient).clamp(-127, 127), scale


def _exact_route(case, s):
    E, k, S = case["experts"], case["top_k"], case["seqs"]
    logits = s["logits"].double()
    lse = torch.logsumexp(logits, dim=1)
    p = torch.exp(logits - lse[:, None])
    keep = torch.ones_like(lse, dtype=torch.bool) if s["mask"] is None else s["mask"].bool()
    ends = s["offsets"].tolist()
    spans = [torch.arange(ends[i], ends[i + 1], device="cuda") for i in range(S)]
    spans = [t[keep[t]] for t in spans]
    filled = sum(1 for t in spans if t.numel())
    total = sum(t.numel() for t in spans)
    counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
    prob_sums = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    dlogits = torch.zeros_like(logits)
    balance = torch.zeros((), dtype=torch.float64, device="cuda")
    for i, t in enumerate(spans):
        n = t.numel()
        if n == 0:
            continue
        counts[i] = torch.bincount(s["ids"][t].reshape(-1).long(), minlength=E).to(torch.int32)
        prob_sums[i] = p[t].sum(dim=0)
        share = E * counts[i].double() / (k * n)
        balance += s["balance"] / filled * torch.dot(share, prob_sums[i] / n)
        # d/dl of sum_e share_e p_e / n is p (share - <share, p>) / n
        toward = share[None, :] - (p[t] @ share)[:, None]
        dlogits[t] = float(s["grads"][0]) * s["balance"] / filled / n * p[t] * toward
        dlogits[t] += float(s["grads"][1]) * s["z"] / total * 2.0 * lse[t][:, None] * p[t]
        w, g = s["probs"][t].double(), s["dprobs"][t].double()
        part = torch.zeros((n, E), dtype=torch.float64, device="cuda")
        part.scatter_(1, s["ids"][t].long(), w * g - w * torch.einsum("tj,tj->t", w, g)[:, None])
        dlogits[t] += part
    z = s["z"] / max(total, 1) * lse[keep].square().sum()
    lse = lse.masked_fill(~keep, -math.inf)
    return {"counts": counts, "prob_sums": prob_sums, "lse": lse, "losses": torch.stack([balance, z]), "dlogits": dlogits}


def _exact_moe(case, s):
    F, E = case["ffn"], case["experts"]
    xq, xs = _exact_codes(s["x"])
    out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not t.numel():
            continue
        pre = (xq[t] @ s["w1q"][e].double().T) * torch.outer(xs[t], s["w1s"][e].double())
        gate, up = pre.split(F, dim=1)
        # the SwiGLU row is held in bf16 before it is quantised for the down product
        hq, hs = _exact_codes((gate * torch.sigmoid(gate) * up).to(torch.bfloat16))
        y = (hq @ s["w2q"][e].double().T) * torch.outer(hs, s["w2s"][e].double())
        out.index_add_(0, t, y * s["probs"][t, j].double()[:, None])
    return out
