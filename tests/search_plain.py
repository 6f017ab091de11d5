"""Plain 64-bit forms of the experts' products, a beam search's step and the caches that follow its beams, written from
their definitions on the CPU, and the bounds that their results are held to.  Test infrastructure only."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}  # half of the smallest step


def ranges(offsets, rows):
    bound = [min(max(int(o), 0), rows) for o in offsets]
    return [(a, max(a, b)) for a, b in zip(bound, bound[1:])]


def products(xs, w, offsets, dys=None):
    """ys, dxs and dw in 64 bits, each with the sum of its terms' magnitudes and their greatest number."""
    xs, w = xs.double().cpu(), w.double().cpu()
    dys = None if dys is None else dys.double().cpu()
    rows, (experts, n, m) = xs.shape[0], w.shape
    ys, dxs, dw = torch.zeros(2, rows, m).double(), torch.zeros(2, rows, n).double(), torch.zeros(2, experts, n, m).double()
    longest = 1
    for e, (a, b) in enumerate(ranges(offsets.tolist(), rows)):
        longest = max(longest, b - a)
        ys[0, a:b], ys[1, a:b] = xs[a:b] @ w[e], xs[a:b].abs() @ w[e].abs()
        if dys is not None:
            dxs[0, a:b], dxs[1, a:b] = dys[a:b] @ w[e].t(), dys[a:b].abs() @ w[e].t().abs()
            dw[0, e], dw[1, e] = xs[a:b].t() @ dys[a:b], xs[a:b].t().abs() @ dys[a:b].abs()
    return (*ys, n), (*dxs, m), (*dw, longest)


def check_product(got, want, what=""):
    """An fp32 sum of n products (exact in fp32, or added without a rounding of their own) errs by at most n steps of 2^-23
    of the sum of their magnitudes: n additions that may round or cut each step; its one rounding to the type by half a
    step."""
    ref, size, n = want
    bound = HALF[got.dtype] * ref.abs() + LEAST[got.dtype] + (1 + HALF[got.dtype]) * n * 2.0 ** -23 * size
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at " \
                          f"{bad.nonzero()[0].tolist()}: {float(err[bad][0])} > {float(bound[bad][0])}"


def continuations(logits, scores, ended=None, end_token=None):
    """The 64-bit score of every continuation, [batch, beams, vocab]; -inf: none."""
    x, scores = logits.double().cpu(), scores.double().cpu()
    batch, beams, vocab = x.shape
    out = torch.full((batch, beams, vocab), -math.inf, dtype=torch.float64)
    for b in range(batch):
        for i in range(beams):
            s, row = float(scores[b, i]), x[b, i]
            if not math.isfinite(s):
                continue
            if ended is not None and bool(ended[b, i]):
                out[b, i, end_token] = s
                continue
            top = float(row.max())  # NaN if any is
            if math.isnan(top) or top == -math.inf:
                continue
            if top == math.inf:
                inf = row == math.inf
                out[b, i] = torch.where(inf, s - math.log(int(inf.sum())), -math.inf)
            else:
                out[b, i] = s + (row - top) - torch.log(torch.exp(row - top).sum())
    return out


# The sum of exponentials: each term to 2^-23 by its function and 2^-24 |d| by its argument d below 0 (d e^d > -0.4, of a
# sum that is at least 1), and at most 40 fp32 additions in a row to 2^-24 each: 48 2^-24 of the sum, or of its logarithm.
LSE = 48 * 2.0 ** -24


def check_selection(got, all_scores, logits, k):
    """The k best of all_scores [batch, beams, vocab] up to what the 32-bit sum allows, equal ones by place."""
    scores, parents, tokens = (x.cpu() for x in got)
    batch, beams, vocab = all_scores.shape
    assert scores.dtype == torch.float32 and parents.dtype == torch.int32 and tokens.dtype == torch.int32
    assert scores.shape == parents.shape == tokens.shape == (batch, k)
    for b in range(batch):
        flat = all_scores[b].flatten()
        want = torch.sort(flat, descending=True, stable=True)
        n = min(k, int((flat > -math.inf).sum()))
        assert (scores[b, n:] == -math.inf).all() and (parents[b, n:] == -1).all() and (tokens[b, n:] == -1).all()
        assert (parents[b, :n] >= 0).all() and (parents[b, :n] < beams).all()
        assert (tokens[b, :n] >= 0).all() and (tokens[b, :n] < vocab).all()
        place = parents[b, :n].long() * vocab + tokens[b, :n].long()
        assert len(set(place.tolist())) == n
        theirs = flat[place]
        assert (theirs - want.values[:n]).abs().max() <= 2 * LSE if n else True  # none that is clearly better is left out
        assert ((scores[b, :n].double() - theirs).abs() <= LSE + 2.0 ** -24 * theirs.abs()).all()
        assert (scores[b, 1:n] <= scores[b, :max(n - 1, 0)][:n - 1]).all() if n else True
        # of one beam, equal logits come in the order of the tokens, and the first of them first
        for i in set(parents[b, :n].tolist()):
            mine = tokens[b, :n][parents[b, :n] == i].long()
            row = all_scores[b, i]
            key = [(-float(row[t]), int(t)) for t in mine]
            assert key == sorted(key)
            first = torch.sort(row, descending=True, stable=True).indices[:len(mine)]
            assert first.tolist() == mine.tolist()
        # where neighbours are clearly apart, the order is the reference's
        full = want.values[:n + 1]
        gap = torch.cat([torch.tensor([math.inf]).double(), full[:-1] - full[1:], torch.tensor([math.inf]).double()])
        for j in range(n):
            if gap[j] > 4 * LSE and (gap[j + 1] > 4 * LSE or j == n - 1 and len(full) == n):
                assert int(place[j]) == int(want.indices[j])


def reorder(state, parents, lengths):
    """What the arrays of `state` (dict of [searches * beams, heads, capacity, ...]) and the lengths become."""
    beams, out = parents.shape[1], {n: x.clone() for n, x in state.items()}
    after = []
    for i, p in enumerate(parents.flatten().tolist()):
        if not 0 <= p < beams:
            after.append(0)
            continue
        source = i // beams * beams + p
        capacity = next(iter(state.values())).shape[2]
        m = min(max(int(lengths[source]), 0), capacity)
        after.append(m)
        for n in out:
            out[n][i, :, :m] = state[n][source, :, :m]
    return out, torch.tensor(after, dtype=torch.int32)
