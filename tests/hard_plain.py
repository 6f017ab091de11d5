"""Plain 64-bit forms of the hard selections (routing, dispatch, cache attention, eviction), written row by row from
their definitions on the CPU.  Test infrastructure only."""
import math

import torch




def route(x, k, bias=None, score="softmax", groups=1, top_groups=None, renormalise=True, scale=1.0):
    """weights, chosen and the scores of every row; x float64 [tokens, experts]."""
    tokens, experts = x.shape
    top_groups = groups if top_groups is None else top_groups
    weights, chosen = torch.zeros(tokens, k, dtype=torch.float64), torch.full((tokens, k), -1, dtype=torch.int32)
    scores = torch.zeros_like(x)
    for t in range(tokens):
        row = x[t].tolist()
        nan = any(math.isnan(v) for v in row)
        row = [-math.inf if math.isnan(v) else v for v in row]
        if score == "softmax":
            m = max(row)
            e = [0.0 if v == -math.inf else (1.0 if v == m else math.exp(v - m)) for v in row]
            total = sum(e)
            s = [v / total if total > 0 else 0.0 for v in e]
        else:
            s = [0.0 if v == -math.inf else 1.0 / (1.0 + math.exp(min(-v, 700.0))) for v in row]
        c = [-math.inf if row[i] == -math.inf else s[i] + (float(bias[i]) if bias is not None else 0.0)
             for i in range(experts)]
        c = [-math.inf if math.isnan(v) else v for v in c]
        if groups > 1:
            size = experts // groups
            best = [sum(sorted(c[g * size:(g + 1) * size], reverse=True)[:2]) for g in range(groups)]
            taken = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            c = [v if i // size in taken else -math.inf for i, v in enumerate(c)]
        first = [i for i in sorted(range(experts), key=lambda i: (-c[i], i)) if c[i] > -math.inf][:k]
        total = sum(s[i] for i in first) if renormalise else 1.0
        for j, i in enumerate(first):
            chosen[t, j] = i
            weights[t, j] = scale * s[i] / total if total > 0 else 0.0
        if nan:
            weights[t] = math.nan
        scores[t] = torch.tensor(s, dtype=torch.float64)
    return weights, chosen, scores


def route_weights(x, chosen, score, renormalise, scale):
    """The weights as a smooth function of the logits, the choice held fixed (for differences and autograd)."""
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    picked = s.gather(1, chosen.clamp(min=0).long()) * (chosen >= 0)
    return scale * picked / picked.sum(1, keepdim=True) if renormalise else scale * picked


def plan(chosen, experts):
    tokens, k = chosen.shape
    by = [[] for _ in range(experts)]
    for pair, e in enumerate(chosen.flatten().tolist()):
        if 0 <= e < experts:
            by[e].append(pair)
    order = [p for rows in by for p in rows]
    offsets = [0]
    for rows in by:
        offsets.append(offsets[-1] + len(rows))
    slot = torch.full((tokens * k,), -1, dtype=torch.int32)
    for at, p in enumerate(order):
        slot[p] = at
    order += [-1] * (tokens * k - len(order))
    return (torch.tensor(offsets, dtype=torch.int32), slot.view(tokens, k), torch.tensor(order, dtype=torch.int32))


def attend(q, k, v, lengths, scale):
    """out, the added weights [batch, heads, capacity], and sum p |v| (for error bounds); all float64."""
    batch, news, q_heads, width = q.shape
    heads, capacity = k.shape[1], k.shape[2]
    group = q_heads // heads
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    added = torch.zeros(batch, heads, capacity, dtype=torch.float64)
    for b in range(batch):
        n = max(0, min(capacity, int(lengths[b])))
        for i in range(news):
            see = n - news + i + 1
            if see <= 0:
                continue
            for j in range(q_heads):
                h = j // group
                p = torch.softmax(k[b, h, :see] @ q[b, i, j] * scale, 0)
                out[b, i, j] = p @ v[b, h, :see]
                size[b, i, j] = p @ v[b, h, :see].abs()
                added[b, h, :see] += p
    return out, added, size


def evict(account, positions, lengths, keep, next_position=None, sinks=0, recent=0):
    """kept and the new lengths."""
    batch, heads, capacity = account.shape
    kept = torch.full((batch, heads, keep), -1, dtype=torch.int32)
    after = []
    for b in range(batch):
        n = max(0, min(capacity, int(lengths[b])))
        m = min(n, keep)
        after.append(m)
        for h in range(heads):
            def rank(i):
                p, x = int(positions[b, h, i]), float(account[b, h, i])
                safe = p < sinks or (recent > 0 and p >= int(next_position[b]) - recent)
                return (0 if safe else 1, 0.0 if safe else (math.inf if math.isnan(x) else -x),
                        0 if safe or not math.isnan(x) else 1, i)
            stays = set(sorted(range(n), key=rank)[:m])
            movers = iter(sorted(i for i in stays if i >= m))
            for i in range(m):
                kept[b, h, i] = i if i in stays else next(movers)
    return kept, torch.tensor(after, dtype=torch.int32)
