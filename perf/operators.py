"""What is measured of the hard selections beside the soft top-k: routing of tokens to experts, their dispatch to
the experts and back, and a cache whose entries are kept by the attention weight that they received.

``own`` chooses between the operators' plain forms (elementary torch operations in 32 bits, rounded once at the
end) and the library's entry points.  A case is a dict of plain values; its "op" names the operator:

  route     scores of a router's logits, the chosen experts and their weights; with "train" the logits' gradient too
  dispatch  the expert order of the chosen pairs, token rows laid out in it, the experts' outputs summed back; with
            "train" the gradients of both too
  attend    new tokens' attention over a cache, with the weight that each entry received added to its account
  evict     the entries of the highest account stay, up to a budget; the survivors fill the holes
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decode step of 16 requests through a router with a balance bias and limited groups: latency
        dict(name="route step 16x256", op="route", tokens=16, experts=256, padded=0, k=8, dtype="bf16", score="sigmoid",
             bias=True, groups=8, top_groups=4, renormalise=True, scale=2.5, train=False),
        # the routing batch of the benchmark (16384 rows of 256 scores, budget 8), fp32 logits, inference
        dict(name="route batch 16384x256", op="route", tokens=16384, experts=256, padded=0, k=8, dtype="fp32",
             score="softmax", bias=False, groups=1, top_groups=1, renormalise=True, scale=1.0, train=False),
        # a training batch with bias and groups, forward and backward
        dict(name="route train 32768x256", op="route", tokens=32768, experts=256, padded=0, k=8, dtype="bf16",
             score="sigmoid", bias=True, groups=8, top_groups=4, renormalise=True, scale=2.5, train=True),
        # a ragged training batch over 60 experts padded to 64, softmax weights left as they are
        dict(name="route train 5003x64", op="route", tokens=5003, experts=64, padded=4, k=6, dtype="fp32",
             score="softmax", bias=False, groups=1, top_groups=1, renormalise=False, scale=1.0, train=True),
        # one decode step of 24 requests to their experts and back
        dict(name="dispatch step 24x2048", op="dispatch", tokens=24, experts=256, k=8, width=2048, dtype="bf16",
             train=False),
        # a training batch to its experts and back, with both gradients
        dict(name="dispatch train 8192x2048", op="dispatch", tokens=8192, experts=256, k=8, width=2048, dtype="bf16",
             train=True),
        # one request's decode step over a short cache: latency
        dict(name="attend 1x1000", op="attend", batch=1, new=1, heads=32, kv_heads=8, width=128, capacity=1024,
             shortest=1000, longest=1000, dtype="bf16"),
        # a serving batch's decode step, requests of mixed length
        dict(name="attend 64x8192 mixed", op="attend", batch=64, new=1, heads=32, kv_heads=8, width=128, capacity=8192,
             shortest=512, longest=8192, dtype="bf16"),
        # one long document
        dict(name="attend 1x200001", op="attend", batch=1, new=1, heads=64, kv_heads=8, width=128, capacity=200064,
             shortest=200001, longest=200001, dtype="fp16"),
        # the last tokens of a prompt as the window that the entries are judged by before the first eviction
        dict(name="attend window 32 of 16384", op="attend", batch=2, new=32, heads=32, kv_heads=8, width=128,
             capacity=16384, shortest=16000, longest=16384, dtype="bf16"),
        # the steady state of a serving batch: one entry over the budget leaves each cache
        dict(name="evict step 32x4097", op="evict", batch=32, kv_heads=8, width=128, capacity=4104, shortest=4097,
             longest=4097, keep=4096, sinks=4, recent=256, dtype="bf16"),
        # after a long prompt: a quarter of its entries stay
        dict(name="evict prompt 131072", op="evict", batch=1, kv_heads=8, width=128, capacity=131072, shortest=130001,
             longest=130001, keep=32768, sinks=4, recent=512, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "attend", "attend", "evict"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log_int(rng, 4, 256 // groups)
        top_groups = rng.randint(max(1, groups // 4), groups)
        renormalise = rng.random() < 0.5  # one renormalised weight is a constant: nothing to learn there
        k = rng.randint(2 if renormalise else 1, min(16, experts // groups * top_groups))
        padded = rng.choice([0, 0, min(3, experts - k)]) if groups == 1 else 0
        return dict(op=op, tokens=_log_int(rng, 1, 32768), experts=experts, padded=padded, k=k,
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=groups > 1 or rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    renormalise=renormalise, scale=rng.choice([1.0, 2.5]), train=rng.random() < 0.5)
    if op == "dispatch":
        width = 8 * _log_int(rng, 16, 512)
        k = rng.randint(1, 8)
        dtype = rng.choice(["fp32", "bf16", "fp16"])
        size = 4 if dtype == "fp32" else 2
        most = min(16384, 8192 * 8 * 2048 * 2 // (k * width * size))
        return dict(op=op, tokens=_log_int(rng, 1, most), experts=_log_int(rng, 8, 256), k=k, width=width, dtype=dtype,
                    train=rng.random() < 0.5)
    width = rng.choice([64, 96, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "attend":
        group = rng.choice([1, 4, 5, 8, 16])
        new = rng.choice([1, 1, 1, 2, rng.randint(3, 32)])
        longest = _log_int(rng, 100, 200000)
        most = 64 * 8192 * 8 * 128 // (2 * longest * kv_heads * width)
        if new > 1:  # no more products than the largest listed window, and none that the plain form cannot hold
            most = min(most, 2 * 32 * 32 * 16384 * 128 // (new * group * kv_heads * longest * width))
        if most < 1:
            new, group, kv_heads, most = 1, min(group, 8), 1, 4
        batch = _log_int(rng, 1, max(1, min(64, most)))
        return dict(op=op, batch=batch, new=new, heads=group * kv_heads, kv_heads=kv_heads, width=width,
                    capacity=longest + rng.randint(0, 63), shortest=max(1, longest // rng.choice([1, 2, 10])),
                    longest=longest, dtype=rng.choice(["bf16", "fp16"]))
    longest = _log_int(rng, 100, 130001)
    most = 130001 * 8 * 128 // (longest * kv_heads * width)
    batch = _log_int(rng, 1, max(1, min(64, most)))
    keep = max(1, longest - rng.choice([1, 16, longest // 4, longest // 2, longest * 3 // 4]))
    return dict(op=op, batch=batch, kv_heads=kv_heads, width=width, capacity=longest + rng.randint(0, 31),
                shortest=max(1, min(longest, keep - rng.randint(0, 9))) if rng.random() < 0.5 else longest,
                longest=longest, keep=keep, sinks=rng.choice([0, 4]), recent=min(keep // 4, 256),
                dtype=rng.choice(["bf16", "fp16"]))


# ------------------------------------------------------------------ inputs
def _masked_groups(c, groups, top_groups):
    """c with the experts of the groups that are not taken at -inf; a group counts by the sum of its best two."""
    if groups == 1:
        return c
    t, e = c.shape
    two = torch.sort(c.view(t, groups, e // groups), dim=2, descending=True).values[:, :, :2].sum(2)
    taken = torch.sort(two, dim=1, descending=True, stable=True).indices[:, :top_groups]
    open_ = torch.zeros(t, groups, dtype=torch.bool, device=c.device).scatter_(1, taken, True)
    return c.masked_fill(~open_.repeat_interleave(e // groups, 1), -math.inf)


def _settled(logits, case, bias):
    """Rows whose choice does not hang on the last bits of a 32-bit score: in 64 bits, neighbours among the first
    k + 1 scores, and the last group taken and the first one left, are equal or at least 4e-6 apart."""
    x = logits.double()
    s = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    c = (s if bias is None else s + bias.double()).masked_fill(x == -math.inf, -math.inf)

    def apart(v):
        gap = (v[:, :-1] - v[:, 1:]).nan_to_num(nan=1.0, posinf=1.0)
        return ((gap == 0) | (gap > 4e-6 * v[:, :-1].abs().nan_to_num(posinf=1.0).clamp(1e-3, 1.0))).all(1)

    g, tg = case["groups"], case["top_groups"]
    ok = apart(torch.sort(_masked_groups(c, g, tg), dim=1, descending=True).values[:, :case["k"] + 1])
    if g > 1 and tg < g:
        t, e = c.shape
        two = torch.sort(c.view(t, g, e // g), dim=2, descending=True).values[:, :, :2].sum(2)
        two = torch.sort(two, dim=1, descending=True).values
        ok &= apart(two[:, tg - 1:tg + 1])
    return ok


def _route_inputs(case, gen):
    t, e = case["tokens"], case["experts"]
    popular = 0.5 * torch.randn(e, generator=gen, device=DEV)
    bias = 0.05 * torch.randn(e, generator=gen, device=DEV) if case["bias"] else None

    def logits(rows):
        x = (torch.randn(rows, e, generator=gen, device=DEV) * 1.5 + popular).to(DTYPES[case["dtype"]])
        if case["padded"]:
            x[:, e - case["padded"]:] = -math.inf
        return x

    x, spare = logits(t), logits(64)
    spare = spare[_settled(spare, case, bias)]
    bad = torch.nonzero(~_settled(x, case, bias))[:, 0]
    x[bad] = spare[torch.arange(len(bad), device=DEV) % len(spare)]
    return dict(case=case, logits=x, bias=bias,
                dweights=torch.randn(t, case["k"], generator=gen, device=DEV) if case["train"] else None)


def _dispatch_inputs(case, gen):
    t, e, k, d, dt = case["tokens"], case["experts"], case["k"], case["width"], DTYPES[case["dtype"]]
    score = torch.randn(t, e, generator=gen, device=DEV) + 0.5 * torch.randn(e, generator=gen, device=DEV)
    top = torch.topk(score, k, dim=1)
    state = dict(case=case, experts=top.indices.int(), weights=torch.softmax(top.values, 1),
                 x=torch.randn(t, d, generator=gen, device=DEV).to(dt),
                 ys=torch.randn(t * k, d, generator=gen, device=DEV).to(dt))
    if case["train"]:
        state["dy"] = torch.randn(t, d, generator=gen, device=DEV).to(dt)
        state["dxs"] = torch.randn(t * k, d, generator=gen, device=DEV).to(dt)
    return state


def _lengths(case, gen):
    b, lo, hi = case["batch"], case["shortest"], case["longest"]
    n = (lo + (hi - lo + 1) * torch.rand(b, generator=gen, device=DEV)).int().clamp(lo, hi)
    n[0] = hi
    return n


def _attend_inputs(case, gen):
    b, m, h, hk, d, s = (case[n] for n in ("batch", "new", "heads", "kv_heads", "width", "capacity"))
    dt = DTYPES[case["dtype"]]
    q = (2.0 * torch.randn(b, m, h, d, generator=gen, device=DEV)).to(dt)
    k = torch.randn(b, hk, s, d, generator=gen, device=DEV, dtype=dt)
    v = torch.randn(b, hk, s, d, generator=gen, device=DEV, dtype=dt)
    acc = torch.rand(b, hk, s, generator=gen, device=DEV)
    return dict(case=case, q=q, k=k, v=v, lengths=_lengths(case, gen), acc=acc, acc_out=torch.zeros_like(acc))


def _evict_inputs(case, gen):
    b, hk, d, s = (case[n] for n in ("batch", "kv_heads", "width", "capacity"))
    dt = DTYPES[case["dtype"]]
    k = torch.randn(b, hk, s, d, generator=gen, device=DEV, dtype=dt)
    v = torch.randn(b, hk, s, d, generator=gen, device=DEV, dtype=dt)
    acc = torch.exp(2.0 * torch.randn(b, hk, s, generator=gen, device=DEV))
    acc[torch.rand(b, hk, s, generator=gen, device=DEV) < 0.05] = 0.0  # entries that were never looked at
    # the positions that are left after earlier evictions: each cache a random part of twice its length, in the
    # order that moves into the holes left
    positions = torch.argsort(torch.rand(b, hk, 2 * s, generator=gen, device=DEV), dim=2)[:, :, :s].int()
    lengths = _lengths(case, gen)
    next_position = torch.full((b,), 2 * s, dtype=torch.int32, device=DEV)
    return dict(case=case, k=k, v=v, acc=acc, positions=positions, lengths=lengths, next_position=next_position,
                acc_out=torch.zeros_like(acc), positions_out=torch.zeros_like(positions))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"route": _route_inputs, "dispatch": _dispatch_inputs, "attend": _attend_inputs,
            "evict": _evict_inputs}[case["op"]](case, gen)


# ------------------------------------------------------------- plain forms
def _plain_route(case, logits, bias, dweights):
    x = logits.float()
    s = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    c = (s if bias is None else s + bias).masked_fill(x == -math.inf, -math.inf)
    c = _masked_groups(c, case["groups"], case["top_groups"])
    top = torch.sort(c, dim=1, descending=True, stable=True)
    there = top.values[:, :case["k"]] > -math.inf
    experts = top.indices[:, :case["k"]]
    chosen = torch.where(there, s.gather(1, experts), 0.0)
    total = chosen.sum(1, keepdim=True) if case["renormalise"] else torch.ones_like(chosen[:, :1])
    weights = case["scale"] * chosen / total
    out = dict(weights=weights, experts=torch.where(there, experts, -1).int())
    if dweights is not None:
        dw = case["scale"] * torch.where(there, dweights, 0.0) / total
        if case["renormalise"]:
            dw = dw - (dw * chosen).sum(1, keepdim=True) / total
        ds = torch.zeros_like(s).scatter_add_(1, experts, torch.where(there, dw, 0.0))
        if case["score"] == "softmax":
            dx = s * (ds - (ds * s).sum(1, keepdim=True))
        else:
            dx = ds * s * (1 - s)
        out["dlogits"] = dx.to(logits.dtype)
    return out


def _plain_dispatch(state):
    case, k, e = state["case"], state["case"]["k"], state["case"]["experts"]
    flat = state["experts"].reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    slot = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=DEV))
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.bincount(flat, minlength=e).cumsum(0)])
    slot2, w = slot.view(-1, k), state["weights"]
    xs = state["x"][order // k]
    picked = state["ys"][slot2].float()
    out = dict(offsets=offsets.int(), slot=slot2.int(), order=order.int(), xs=xs,
               y=(picked * w[:, :, None]).sum(1).to(xs.dtype))
    if case["train"]:
        dy = state["dy"].float()
        out["dys"] = (dy[order // k] * w.reshape(-1)[order][:, None]).to(xs.dtype)
        out["dweights"] = (picked * dy[:, None, :]).sum(2)
        out["dx"] = state["dxs"][slot2].float().sum(1).to(xs.dtype)
    return out


def _plain_attend(state):
    case, q, k, v, lengths = (state[n] for n in ("case", "q", "k", "v", "lengths"))
    b, m, h, d = q.shape
    hk, s = k.shape[1], k.shape[2]
    rows = q.float().view(b, m, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, m * (h // hk), d)
    logits = torch.matmul(rows, k.float().transpose(2, 3)).view(b, hk, m, h // hk, s) / math.sqrt(d)
    entry = torch.arange(s, device=DEV)
    last = lengths.long()[:, None] - m + torch.arange(m, device=DEV)  # the last entry that a new token sees
    seen = (entry <= last[:, :, None])[:, None, :, None, :]
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(4, keepdim=True)
    p = torch.exp(logits - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(4, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    out = torch.matmul(p.view(b, hk, m * (h // hk), s), v.float())
    out = out.view(b, hk, m, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, m, h, d).to(q.dtype)
    there = (entry < lengths[:, None])[:, None, :]
    return dict(out=out, acc=torch.where(there, state["acc"] + p.sum((2, 3)), state["acc_out"]))


def _plain_evict(state):
    case, acc, positions = state["case"], state["acc"], state["positions"]
    b, hk, s = acc.shape
    keep = case["keep"]
    entry = torch.arange(s, device=DEV).expand(b, hk, s)
    lengths = state["lengths"].long()[:, None, None]
    after = torch.clamp(lengths, max=keep)
    there = entry < lengths
    safe = (positions < case["sinks"]) | (positions >= state["next_position"][:, None, None] - case["recent"])
    rank = torch.where(safe, math.inf, acc).masked_fill(~there, -math.inf)
    first = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :keep]
    stays = torch.zeros_like(there).scatter_(2, first, True) & there
    hole = ~stays & (entry < after)
    mover = stays & (entry >= after)
    # the n-th hole takes the n-th survivor from behind the budget
    movers = torch.sort(torch.where(mover, entry, s), dim=2).values
    nth = (hole.long().cumsum(2) - 1).clamp(min=0)
    kept = torch.where(hole, movers.gather(2, nth), entry)[:, :, :keep]
    filled = entry[:, :, :keep] < after
    source = torch.where(filled, kept, entry[:, :, :keep])
    wide = source[..., None].expand(-1, -1, -1, case["width"])
    state["k"][:, :, :keep] = state["k"].gather(2, wide)
    state["v"][:, :, :keep] = state["v"].gather(2, wide)
    state["acc_out"][:, :, :keep] = torch.where(filled, acc.gather(2, source), state["acc_out"][:, :, :keep])
    state["positions_out"][:, :, :keep] = torch.where(filled, positions.gather(2, source),
                                                      state["positions_out"][:, :, :keep])
    return dict(kept=torch.where(filled, kept, -1).int(), lengths=after[:, 0, 0].int(), k=state["k"], v=state["v"],
                acc=state["acc_out"], positions=state["positions_out"])


# --------------------------------------------------------------- one pass
def _own_route(state):
    import sparse_selection_primitive_amd as L
    case = state["case"]
    kinds = dict(score=case["score"], renormalise=case["renormalise"], scale=case["scale"])
    weights, experts = L.route_forward(state["logits"], case["k"], state["bias"], groups=case["groups"],
                                       top_groups=case["top_groups"], **kinds)
    out = dict(weights=weights, experts=experts)
    if case["train"]:
        out["dlogits"] = L.route_backward(state["dweights"], state["logits"], experts, **kinds)
    return out


def _own_dispatch(state):
    import sparse_selection_primitive_amd as L
    case = state["case"]
    offsets, slot, order = L.dispatch_plan(state["experts"], case["experts"])
    out = dict(offsets=offsets, slot=slot, order=order, xs=L.dispatch_forward(state["x"], slot, offsets),
               y=L.combine_forward(state["ys"], slot, state["weights"]))
    if case["train"]:
        out["dys"], out["dweights"] = L.combine_backward(state["dy"], state["ys"], slot, state["weights"], offsets)
        out["dx"] = L.dispatch_backward(state["dxs"], slot)
    return out


def _own_attend(state):
    import sparse_selection_primitive_amd as L
    out = L.cache_attend(state["q"], state["k"], state["v"], state["lengths"], state["acc"],
                         account_out=state["acc_out"])
    return dict(out=out, acc=state["acc_out"])


def _own_evict(state):
    import sparse_selection_primitive_amd as L
    case = state["case"]
    kept, lengths = L.cache_evict(state["k"], state["v"], state["acc"], state["positions"], state["lengths"],
                                  case["keep"], next_position=state["next_position"], sinks=case["sinks"],
                                  recent=case["recent"], account_out=state["acc_out"],
                                  positions_out=state["positions_out"])
    return dict(kept=kept, lengths=lengths, k=state["k"], v=state["v"], acc=state["acc_out"],
                positions=state["positions_out"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "dispatch": _own_dispatch, "attend": _own_attend, "evict": _own_evict}[op](state)
    if op == "route":
        return _plain_route(state["case"], state["logits"], state["bias"], state["dweights"])
    return {"dispatch": _plain_dispatch, "attend": _plain_attend, "evict": _plain_evict}[op](state)


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        moved = t * e * size + t * k * 8 + (4 * e if case["bias"] else 0)
        if case["train"]:
            moved += t * k * 4 + t * e * size
        return {"bytes": moved, "flops": t * e * (8 if case["train"] else 4)}
    if op == "dispatch":
        t, k, d = case["tokens"], case["k"], case["width"]
        moved = t * k * 8 + 8 * t * k + 4 * (case["experts"] + 1) + (2 * t * d + 2 * t * k * d) * size
        if case["train"]:
            moved += (2 * t * d + 2 * t * k * d) * size + t * k * 4
        return {"bytes": moved, "flops": 2 * t * k * d * (3 if case["train"] else 1)}
    if op == "attend":
        # lengths lie evenly between the shortest and the longest; the first is the longest
        b, lo, hi = case["batch"], case["shortest"], case["longest"]
        entries = hi + (b - 1) * (lo + hi) // 2
        hk, d, rows = case["kv_heads"], case["width"], case["new"] * case["heads"]
        return {"bytes": entries * hk * (2 * d * size + 8) + 2 * b * rows * d * size,
                "flops": 4 * entries * rows * d}
    b, lo, hi = case["batch"], case["shortest"], case["longest"]
    entries = hi + (b - 1) * (lo + hi) // 2
    gone = sum(max(0, n - case["keep"]) for n in [hi] + [(lo + hi) // 2] * (b - 1))
    # an entry behind the budget stays with the chance that any does, and moves once
    moved = gone * case["keep"] // max(1, hi)
    stay = entries - gone
    return {"bytes": case["kv_heads"] * (8 * entries + 12 * stay + moved * 4 * case["width"] * size),
            "flops": entries * case["kv_heads"]}


# ------------------------------------------------------- in 64 bits, apart
def _exact_route(state):
    case = state["case"]
    x = state["logits"].double()
    t, e = x.shape
    k, groups, size = case["k"], case["groups"], case["experts"] // case["groups"]
    if case["score"] == "softmax":
        s = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    c = s.clone()
    if state["bias"] is not None:
        c += state["bias"].double()
    c[torch.isinf(x)] = -math.inf
    rows = torch.arange(t, device=DEV)
    if groups > 1:
        best = torch.topk(c.view(t, groups, size), min(2, size), dim=2).values.sum(2)
        closed = torch.ones(t, groups, dtype=torch.bool, device=DEV)
        for _ in range(case["top_groups"]):
            g = best.argmax(1)
            closed[rows, g] = False
            best[rows, g] = -math.inf
        c.view(t, groups, size)[closed] = -math.inf
    experts = torch.empty(t, k, dtype=torch.long, device=DEV)
    number = torch.arange(e, device=DEV)
    for j in range(k):
        top = c.amax(1, keepdim=True)
        first = torch.where(c == top, number, e).amin(1)
        experts[:, j] = torch.where(top[:, 0] == -math.inf, -1, first)
        c[rows, first] = -math.inf
    there = experts >= 0
    chosen = torch.where(there, s[rows[:, None], experts.clamp(min=0)], 0.0)
    total = chosen.sum(1, keepdim=True) if case["renormalise"] else torch.ones(t, 1, dtype=torch.double, device=DEV)
    out = dict(weights=case["scale"] * chosen / total, experts=experts.int())
    if case["train"]:
        g = torch.where(there, state["dweights"].double(), 0.0)
        # d weight_j / d score_i = scale (delta_ij - [renormalised] chosen_j / total) / total
        mean = (g * chosen).sum(1, keepdim=True) / total if case["renormalise"] else 0.0
        per = case["scale"] * (g - mean) / total * chosen
        dx = torch.zeros_like(x)
        for j in range(k):
            i = experts[:, j].clamp(min=0)
            slope = 1.0 if case["score"] == "softmax" else 1.0 - s[rows, i]
            dx[rows, i] += torch.where(there[:, j], per[:, j] * slope, 0.0)
        if case["score"] == "softmax":
            dx -= s * per.masked_fill(~there, 0.0).sum(1, keepdim=True)
        out["dlogits"] = dx
    return out


def _exact_dispatch(state):
    case, k, e = state["case"], state["case"]["k"], state["case"]["experts"]
    flat = state["experts"].reshape(-1).long()
    place = flat * len(flat) + torch.arange(len(flat), device=DEV)  # all different: any sort is stable
    order = torch.argsort(place)
    slot = torch.argsort(order).view(-1, k)
    offsets = torch.searchsorted(flat[order].contiguous(), torch.arange(e + 1, device=DEV))
    w, d = state["weights"].double(), case["width"]
    t = case["tokens"]
    y = torch.zeros(t, d, dtype=torch.double, device=DEV)
    for j in range(k):
        y += w[:, j, None] * state["ys"][slot[:, j]].double()
    out = dict(offsets=offsets.int(), slot=slot.int(), order=order.int(), xs=state["x"][order // k].double(), y=y)
    if case["train"]:
        dy = state["dy"].double()
        dys = torch.empty(t * k, d, dtype=torch.double, device=DEV)
        dw = torch.empty(t, k, dtype=torch.double, device=DEV)
        dx = torch.zeros(t, d, dtype=torch.double, device=DEV)
        for j in range(k):
            dys[slot[:, j]] = w[:, j, None] * dy
            dw[:, j] = (state["ys"][slot[:, j]].double() * dy).sum(1)
            dx += state["dxs"][slot[:, j]].double()
        out.update(dys=dys, dweights=dw, dx=dx)
    return out


def _exact_attend(state):
    case, q, k, v, lengths = (state[n] for n in ("case", "q", "k", "v", "lengths"))
    b, m, h, d = q.shape
    g = h // k.shape[1]
    out = torch.zeros(b, m, h, d, dtype=torch.double, device=DEV)
    acc = state["acc_out"].double()
    for i, n in enumerate(lengths.tolist()):
        for a in range(k.shape[1]):
            keys, values = k[i, a, :n].double(), v[i, a, :n].double()
            acc[i, a, :n] = state["acc"][i, a, :n].double()
            z = q[i, :, a * g:(a + 1) * g].double().reshape(m * g, d) @ keys.T * d ** -0.5
            hidden = torch.arange(n, device=DEV) > n - m + torch.arange(m, device=DEV)[:, None]
            z[hidden.repeat_interleave(g, 0)] = -math.inf
            z = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)).nan_to_num(nan=0.0)
            out[i, :, a * g:(a + 1) * g] = (z @ values).view(m, g, d)
            acc[i, a, :n] += z.sum(0)
    return dict(out=out, acc=acc)


def _exact_evict(state):
    case, keep = state["case"], state["case"]["keep"]
    acc, positions = state["acc"], state["positions"]
    b, hk, s = acc.shape
    kept = torch.full((b, hk, keep), -1, dtype=torch.int32, device=DEV)
    k, v = state["k"], state["v"]
    acc_out, positions_out = state["acc_out"], state["positions_out"]
    after = []
    for i, n in enumerate(state["lengths"].tolist()):
        m = min(n, keep)
        after.append(m)
        for a in range(hk):
            p, r = positions[i, a, :n].long(), acc[i, a, :n].double()
            r[(p < case["sinks"]) | (p >= int(state["next_position"][i]) - case["recent"])] = math.inf
            # by account, and by slot where accounts are equal
            stays = torch.argsort(-r, stable=True)[:m].sort().values
            front = torch.arange(m, device=DEV)
            holes = front[~torch.isin(front, stays)]
            front[holes] = stays[stays >= m]
            kept[i, a, :m] = front.int()
            moved = front[holes]
            k[i, a, holes], v[i, a, holes] = k[i, a, moved], v[i, a, moved]
            acc_out[i, a, :m], positions_out[i, a, :m] = acc[i, a, front], positions[i, a, front]
    return dict(kept=kept, lengths=torch.tensor(after, dtype=torch.int32, device=DEV), k=k, v=v, acc=acc_out,
                positions=positions_out)


def exact(case, seed):
    state = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "attend": _exact_attend,
            "evict": _exact_evict}[case["op"]](state)
