"""What is measured of the operators that join the hard selections into a whole decoder: the experts' products between
dispatch and combine, the selection of a beam search, and the caches that follow its beams.

``own`` chooses between the operators' plain forms (elementary torch operations in 32 bits, in 64 where candidates are
compared, rounded once at the end) and the library's entry points.  A case is a dict of plain values; its "op" names
the operator:

  experts  rows in expert order times their expert's matrix; with "train" the gradients of rows and matrices too
  beams    the best continuations of a beam search over beams and vocabulary
  reorder  every beam's cache becomes that of its parent, in place, with accounts and positions
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decode step of one request: 8 rows, each of another expert; matrices stored [outputs, inputs]
        dict(name="experts step 1", op="experts", tokens=1, experts=256, k=8, inputs=2048, outputs=1024, dtype="bf16",
             stored="out_in", train=False),
        # one decode step of 24 requests: every expert that is met has its matrix read for a row or two
        dict(name="experts step 24", op="experts", tokens=24, experts=256, k=8, inputs=2048, outputs=1024,
             dtype="bf16", stored="in_out", train=False),
        # a training batch over many experts, 256 rows each in the mean, with both gradients
        dict(name="experts train 8192 of 256", op="experts", tokens=8192, experts=256, k=8, inputs=2048, outputs=1024,
             dtype="bf16", stored="in_out", train=True),
        # a ragged training batch over 64 experts, sizes that no tile divides
        dict(name="experts train 5003 of 64", op="experts", tokens=5003, experts=64, k=6, inputs=2056, outputs=1416,
             dtype="fp16", stored="out_in", train=True),
        # a prompt through few wide experts
        dict(name="experts prompt 8192 of 8", op="experts", tokens=8192, experts=8, k=2, inputs=4096, outputs=14336,
             dtype="bf16", stored="in_out", train=False),
        # one request's search step: latency
        dict(name="beams 1x4 of 32000", op="beams", batch=1, beams=4, vocab=32000, padded=0, k=8, ended=0.0,
             dtype="bf16"),
        # a ragged fp32 step with ended beams and a padded vocabulary, twice the beams kept
        dict(name="beams 16x5 of 50021", op="beams", batch=16, beams=5, vocab=50021, padded=27, k=10, ended=0.2,
             dtype="fp32"),
        # a serving batch over a large vocabulary
        dict(name="beams 64x8 of 131072", op="beams", batch=64, beams=8, vocab=131072, padded=0, k=16, ended=0.1,
             dtype="bf16"),
        # one request's beams take over their parents' short caches: latency
        dict(name="reorder 1x4 of 1000", op="reorder", batch=1, beams=4, kv_heads=8, width=128, capacity=1024,
             shortest=1000, longest=1000, account=False, dtype="bf16"),
        # ragged caches with accounts and positions
        dict(name="reorder 12x5 of 3001", op="reorder", batch=12, beams=5, kv_heads=2, width=96, capacity=3003,
             shortest=700, longest=3001, account=True, dtype="fp16"),
        # a serving batch with long caches that are kept within a budget
        dict(name="reorder 16x4 of 8192", op="reorder", batch=16, beams=4, kv_heads=8, width=128, capacity=8192,
             shortest=2048, longest=8192, account=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts", "experts", "beams", "reorder"])
    if op == "experts":
        train = rng.random() < 0.5
        experts, inputs, outputs = _log_int(rng, 4, 256), 8 * _log_int(rng, 32, 512), 8 * _log_int(rng, 32, 1792)
        experts = max(4, min(experts, 256 * 2048 * 1024 // (inputs * outputs)))
        k = rng.randint(1, min(8, experts))
        most = 8192 * 2 * 4096 * 14336 // ((3 if train else 1) * k * inputs * outputs)
        tokens = _log_int(rng, 1, max(1, min(16384, most)))
        while tokens * k * (inputs + outputs) > 65536 * 8192:
            tokens //= 2
        return dict(op=op, tokens=tokens, experts=experts, k=k, inputs=inputs, outputs=outputs,
                    dtype=rng.choice(["bf16", "fp16"]), stored=rng.choice(["in_out", "out_in"]), train=train)
    if op == "beams":
        beams, vocab = rng.randint(1, 16), _log_int(rng, 1000, 200000)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        most = 64 * 8 * 131072 * 2 // (beams * vocab * (4 if dtype == "fp32" else 2))
        return dict(op=op, batch=_log_int(rng, 1, max(1, min(256, most))), beams=beams, vocab=vocab,
                    padded=rng.choice([0, 0, rng.randint(1, 64)]), k=rng.randint(beams, 2 * beams),
                    ended=rng.choice([0.0, 0.2]), dtype=dtype)
    width, kv_heads, beams = rng.choice([64, 96, 128, 256]), rng.choice([1, 2, 4, 8]), rng.randint(2, 12)
    longest = _log_int(rng, 100, 32000)
    most = 16 * 4 * 8 * 4096 * 128 // (longest * kv_heads * width * beams)
    return dict(op=op, batch=_log_int(rng, 1, max(1, min(64, most))), beams=beams, kv_heads=kv_heads, width=width,
                capacity=longest + rng.randint(0, 63), shortest=max(1, longest // rng.choice([1, 2, 10])),
                longest=longest, account=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))


# ------------------------------------------------------------------ inputs
def _expert_inputs(case, gen):
    t, e, k, n, m = (case[x] for x in ("tokens", "experts", "k", "inputs", "outputs"))
    dt = DTYPES[case["dtype"]]
    # popular experts get more rows; some may get none
    score = torch.randn(t, e, generator=gen, device=DEV) + 0.5 * torch.randn(e, generator=gen, device=DEV)
    chosen = torch.topk(score, k, dim=1).indices.reshape(-1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.bincount(chosen, minlength=e).cumsum(0)])
    w = torch.randn(e, *((n, m) if case["stored"] == "in_out" else (m, n)), generator=gen, device=DEV, dtype=dt)
    w *= n ** -0.5
    state = dict(case=case, offsets=offsets.int(), w=w if case["stored"] == "in_out" else w.transpose(1, 2),
                 xs=torch.randn(t * k, n, generator=gen, device=DEV, dtype=dt))
    if case["train"]:
        state["dys"] = torch.randn(t * k, m, generator=gen, device=DEV, dtype=dt)
    return state


def _candidates(state, logits=None, scores=None, ended=None):
    """The 64-bit scores of all continuations, [batch, beams * vocab]."""
    x = (state["logits"] if logits is None else logits).double()
    scores, ended = state["scores"] if scores is None else scores, state["ended"] if ended is None else ended
    logp = x - torch.logsumexp(x, 2, keepdim=True)
    end = torch.zeros(x.shape[2], dtype=torch.double, device=DEV).fill_(-math.inf)
    end[state["end"]] = 0.0
    return (scores.double()[:, :, None] + torch.where(ended[:, :, None], end, logp)).flatten(1)


def _beam_inputs(case, gen):
    b, n, v, dt = case["batch"], case["beams"], case["vocab"], DTYPES[case["dtype"]]

    def draws(rows):
        logits = (3.0 * torch.randn(rows, n, v, generator=gen, device=DEV)).to(dt)
        if case["padded"]:
            logits[:, :, v - case["padded"]:] = -math.inf
        scores = -10.0 * torch.rand(rows, n, generator=gen, device=DEV) - 5.0
        # an ended beam is one that ended well, or it would have been dropped
        ended = torch.rand(rows, n, generator=gen, device=DEV) < case["ended"]
        return logits, torch.sort(scores, dim=1, descending=True).values, ended

    # searches whose order does not hang on the last bits of a 32-bit score: among the best k + 1 continuations
    # neighbours are equal or clearly apart
    state = dict(case=case, end=2)
    parts = []
    for at in range(0, b, 16):
        part = draws(min(16, b - at))
        for _ in range(20):
            top = torch.topk(_candidates(state, *part), min(case["k"] + 1, n * v), dim=1).values
            gap = (top[:, :-1] - top[:, 1:]).nan_to_num(nan=1.0, posinf=1.0)
            bad = ~((gap == 0) | (gap > 3e-5)).all(1)
            if not bool(bad.any()):
                break
            for to, new in zip(part, draws(len(bad))):
                to[bad] = new[bad]
        parts.append(part)
    state["logits"], state["scores"], state["ended"] = (torch.cat(p) for p in zip(*parts))
    return state


def _lengths(case, gen):
    b, n, lo, hi = case["batch"], case["beams"], case["shortest"], case["longest"]
    # the beams of a search are equally long, but for those that ended a while ago
    length = (lo + (hi - lo + 1) * torch.rand(b, 1, generator=gen, device=DEV)).int().clamp(lo, hi).expand(b, n).clone()
    ended = torch.rand(b, n, generator=gen, device=DEV) < 0.1
    length = torch.where(ended, (length - 7).clamp(min=0), length)
    length[0, 0] = hi
    return length.flatten().int()


def _reorder_inputs(case, gen):
    b, n, h, d, s = (case[x] for x in ("batch", "beams", "kv_heads", "width", "capacity"))
    dt = DTYPES[case["dtype"]]
    state = dict(case=case, lengths=_lengths(case, gen),
                 k=torch.randn(b * n, h, s, d, generator=gen, device=DEV, dtype=dt),
                 v=torch.randn(b * n, h, s, d, generator=gen, device=DEV, dtype=dt),
                 parents=torch.randint(0, n, (b, n), generator=gen, device=DEV, dtype=torch.int32))
    if case["account"]:
        state["account"] = torch.rand(b * n, h, s, generator=gen, device=DEV)
        state["positions"] = torch.randint(0, 2 * s, (b * n, h, s), generator=gen, device=DEV, dtype=torch.int32)
    return state


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"experts": _expert_inputs, "beams": _beam_inputs, "reorder": _reorder_inputs}[case["op"]](case, gen)


# ------------------------------------------------------------- plain forms
def _plain_experts(state):
    xs, w = state["xs"], state["w"]
    bounds = state["offsets"].tolist()
    ys = xs.new_empty(xs.shape[0], w.shape[2])
    train = state["case"]["train"]
    if train:
        dys, dxs, dw = state["dys"], torch.empty_like(xs), torch.zeros_like(w)
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            continue
        rows, matrix = xs[a:b].float(), w[e].float()
        ys[a:b] = rows @ matrix
        if train:
            dy = dys[a:b].float()
            dxs[a:b] = dy @ matrix.t()
            dw[e] = rows.t() @ dy
    return dict(ys=ys, dxs=dxs, dw=dw) if train else dict(ys=ys)


def _plain_beams(state):
    case, x = state["case"], state["logits"].float()
    n, v = x.shape[1:]
    top = x.amax(2, keepdim=True)
    logp = x - (top + torch.log(torch.exp(x - top).sum(2, keepdim=True)))
    end = torch.full((v,), -math.inf, device=DEV)
    end[state["end"]] = 0.0
    logp = torch.where(state["ended"][:, :, None], end, logp)
    # one 64-bit key a continuation: the order of its score, then the lowest index
    bits = (state["scores"][:, :, None] + logp).flatten(1).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
    key = order * 2 ** 32 + (2 ** 32 - 1 - torch.arange(n * v, device=DEV))
    first = 2 ** 32 - 1 - (torch.topk(key, case["k"], dim=1).values & 0xffffffff)
    scores = (state["scores"][:, :, None] + logp).flatten(1).gather(1, first)
    there = scores > -math.inf
    return dict(scores=scores, parents=torch.where(there, first // v, -1).int(),
                tokens=torch.where(there, first % v, -1).int())


def _plain_reorder(state):
    case, parents, lengths = state["case"], state["parents"], state["lengths"]
    b, n = parents.shape
    source = (torch.arange(b, device=DEV)[:, None] * n + parents).flatten()
    after = lengths[source]
    there = (torch.arange(case["capacity"], device=DEV) < after[:, None])[:, None, :]
    out = dict(lengths=after)
    for name in ("k", "v", "account", "positions"):
        if name in state:
            x = state[name]
            x.copy_(torch.where(there[..., None] if x.dim() == 4 else there, x[source], x))
            out[name] = x
    return out


# --------------------------------------------------------------- one pass
def _own_experts(state):
    import sparse_selection_primitive_amd as L
    xs, w, offsets = state["xs"], state["w"], state["offsets"]
    out = dict(ys=L.expert_product_forward(xs, w, offsets))
    if state["case"]["train"]:
        out["dxs"], out["dw"] = L.expert_product_backward(state["dys"], xs, w, offsets)
    return out


def _own_beams(state):
    import sparse_selection_primitive_amd as L
    scores, parents, tokens = L.beam_select(state["logits"], state["scores"], state["case"]["k"], ended=state["ended"],
                                            end_token=state["end"])
    return dict(scores=scores, parents=parents, tokens=tokens)


def _own_reorder(state):
    import sparse_selection_primitive_amd as L
    names = [n for n in ("k", "v", "account", "positions") if n in state]
    after = L.cache_reorder(state["k"], state["v"], state["parents"], state["lengths"], state.get("account"),
                            state.get("positions"))
    return dict(lengths=after, **{n: state[n] for n in names})


def run(state):
    op = state["case"]["op"]
    if own:
        return {"experts": _own_experts, "beams": _own_beams, "reorder": _own_reorder}[op](state)
    return {"experts": _plain_experts, "beams": _plain_beams, "reorder": _plain_reorder}[op](state)


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "experts":
        t, e, k, n, m = (case[x] for x in ("tokens", "experts", "k", "inputs", "outputs"))
        rows, met = t * k, e * (1.0 - (1.0 - k / e) ** t)  # experts that are met, if all are as popular
        moved, flops = size * (rows * (n + m) + met * n * m), 2 * rows * n * m
        if case["train"]:
            moved += size * (rows * (n + m) + e * n * m)
            flops *= 3
        return {"bytes": moved, "flops": flops}
    if op == "beams":
        b, n, v, k = (case[x] for x in ("batch", "beams", "vocab", "k"))
        live = b * n * (1.0 - case["ended"])
        return {"bytes": live * v * size + b * (n * 5 + k * 12), "flops": 4 * live * v}
    # parents fall evenly: a beam keeps its cache with 1/n, and a cache is read once however many take it over
    b, n, lo, hi = case["batch"], case["beams"], case["shortest"], case["longest"]
    entries = (hi + (b - 1) * (lo + hi) / 2) * case["kv_heads"]
    written = n - 1
    read = n * (1.0 - (1.0 - 1.0 / n) ** (n - 1))  # some other beam takes it
    per = 2 * case["width"] * size + (8 if case["account"] else 0)
    return {"bytes": entries * per * (written + read) + b * n * 12, "flops": 0}


# ------------------------------------------------------- in 64 bits, apart
def _exact_experts(state):
    case, xs, w = state["case"], state["xs"], state["w"]
    belongs = torch.searchsorted(state["offsets"][1:].long().contiguous(), torch.arange(xs.shape[0], device=DEV),
                                 right=True)
    ys = torch.zeros(xs.shape[0], w.shape[2], dtype=torch.double, device=DEV)
    out = dict(ys=ys)
    if case["train"]:
        out["dxs"] = torch.zeros(xs.shape, dtype=torch.double, device=DEV)
        out["dw"] = torch.zeros(w.shape, dtype=torch.double, device=DEV)
    for e in range(case["experts"]):
        mine = torch.nonzero(belongs == e)[:, 0]
        if len(mine) == 0:
            continue
        rows, matrix = xs[mine].double(), w[e].double().contiguous()
        ys[mine] = torch.mm(rows, matrix)
        if case["train"]:
            dy = state["dys"][mine].double()
            out["dxs"][mine] = torch.mm(dy, matrix.t().contiguous())
            out["dw"][e] = torch.mm(rows.t().contiguous(), dy)
    return out


def _exact_beams(state):
    case = state["case"]
    b, v = case["batch"], case["vocab"]
    out = dict(scores=torch.full((b, case["k"]), -math.inf, dtype=torch.double, device=DEV),
               parents=torch.full((b, case["k"]), -1, dtype=torch.int32, device=DEV),
               tokens=torch.full((b, case["k"]), -1, dtype=torch.int32, device=DEV))
    for at in range(0, b, 16):
        part = slice(at, at + 16)
        c = _candidates(state, state["logits"][part], state["scores"][part], state["ended"][part])
        rows = torch.arange(len(c), device=DEV)
        number = torch.arange(c.shape[1], device=DEV)
        for j in range(case["k"]):
            best = c.amax(1, keepdim=True)
            first = torch.where(c == best, number, c.shape[1]).amin(1)
            there = best[:, 0] > -math.inf
            out["scores"][part, j] = best[:, 0]
            out["parents"][part, j] = torch.where(there, first // v, -1).int()
            out["tokens"][part, j] = torch.where(there, first % v, -1).int()
            c[rows, first] = -math.inf
    return out


def _exact_reorder(state):
    n = state["case"]["beams"]
    lengths, parents = state["lengths"].tolist(), state["parents"].flatten().tolist()
    out = dict(lengths=torch.empty_like(state["lengths"]))
    for name in ("k", "v", "account", "positions"):
        if name in state:
            out[name] = state[name].clone()
    for i, p in enumerate(parents):
        source = i // n * n + p
        m = lengths[source]
        out["lengths"][i] = m
        for name in out:
            if name != "lengths":
                out[name][i, :, :m] = state[name][source, :, :m]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"experts": _exact_experts, "beams": _exact_beams, "reorder": _exact_reorder}[case["op"]](state)
