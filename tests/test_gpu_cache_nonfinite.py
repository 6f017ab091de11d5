"""Infinities and NaN that a token does see: they reach its output, and nothing else.

Each case compares with the same call on finite inputs, bit by bit, wherever the odd value must not show."""
import math

import pytest

import hard_plain as plain

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


def inputs(batch, heads, capacity, width, news, group, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(batch, heads, capacity, width, generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(batch, news, heads * group, width, generator=g, device="cuda").to(dtype)
    return q, k, v


@pytest.mark.parametrize("news", [1, 3])
@pytest.mark.parametrize("group", [1, 4, 16, 17, 32, 40, 70])
@pytest.mark.parametrize("width", [64, 120, 256])
@pytest.mark.parametrize("caches", ["few", "many"])
def test_value_that_the_newest_token_sees(L, caches, width, group, news):
    """The newest entry's value, at lengths on and off a block of 32 and below one, and one in an earlier block."""
    lengths = [1, 5, 31, 32, 33, 64, 77, 96, 250]
    if caches == "many":  # enough for a workgroup each
        lengths = lengths * 29
    batch, capacity = len(lengths), 256
    q, k, v = inputs(batch, 1, capacity, width, news, group)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    account = torch.zeros(batch, 1, capacity, device="cuda")
    clean = L.cache_attend(q, k, v, n, account)
    assert torch.isfinite(clean).all()
    for odd in (math.nan, math.inf, -math.inf):
        for back in (1, 40):
            at = n.long() - back
            rows = torch.nonzero(at >= 0)[:, 0]
            w = v.clone()
            w[rows, 0, at[rows], ::3] = odd
            added = torch.zeros_like(account)
            out = L.cache_attend(q, k, w, n, added)
            seen = torch.zeros(batch, news, group, width, dtype=torch.bool, device="cuda")
            first = news - back if back <= news else 0  # the first token that sees the entry
            for i in range(max(0, first), news):
                seen[rows, i, :, ::3] = True
            assert not torch.isfinite(out[seen]).any()
            assert torch.equal(out[~seen], clean[~seen])
            assert torch.equal(added, account)  # the weights do not depend on the values
            assert torch.equal(torch.isnan(L.cache_attend(q, k, w, n)), torch.isnan(out))


@pytest.mark.parametrize("news,group", [(4, 2), (4, 4), (9, 4), (40, 1)])
@pytest.mark.parametrize("batch,capacity", [(2, 120), (2, 700), (130, 300)])
def test_row_of_nan_gives_to_what_it_sees(L, batch, capacity, news, group):
    """A query of NaN makes the accounts of the entries that its token sees NaN, not those of the newer ones."""
    q, k, v = inputs(batch, 2, capacity, 64, news, group, seed=1)
    n = torch.tensor([capacity, capacity - 37] * (batch // 2), dtype=torch.int32, device="cuda")
    account = torch.rand(batch, 2, capacity, device="cuda")
    bad = q.clone()
    bad[:, 0, 0] = math.nan  # of the first new token, on key head 0
    got = torch.full_like(account, -7.0)
    out = L.cache_attend(bad, k, v, n, account, account_out=got)
    clean = torch.full_like(account, -7.0)
    want = L.cache_attend(q, k, v, n, account, account_out=clean)
    assert torch.isnan(out[:, 0, 0]).all()
    hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    hit[:, 0, 0] = True
    # rows of a tile share the steps at which their bases move, so the others' bits may change: twice the bound of
    # test_gpu_cache, with logits below 16 (delta 7e-5) and a mean |v| below 1.5
    off = (out.float() - want.float()).abs()[~hit]
    assert (off <= 2.0 ** -10 + 2.0 ** -7 * want.float().abs()[~hit]).all()
    entry = torch.arange(capacity, device="cuda")
    sees = entry[None] <= n[:, None] - news  # what the first new token sees
    assert torch.isnan(got[:, 0][sees]).all()
    # a newer entry gets nothing from that row either way
    for a, b in ((got[:, 0][~sees], clean[:, 0][~sees]), (got[:, 1], clean[:, 1])):
        assert ((a - b).abs() <= 2.0 ** -11 * (1.0 + b.abs())).all()


@pytest.mark.parametrize("width", [40, 64, 72, 96, 136, 200])
@pytest.mark.parametrize("news,group", [(2, 4), (7, 3), (20, 4)])
def test_row_of_minus_infinite_logits_gives_nothing(L, width, news, group):
    """A query that makes every logit -inf has no weight: zeros, and the accounts are the other rows' alone."""
    q, k, v = inputs(1, 1, 400, width, news, group, seed=2)
    k[..., 0] = k[..., 0].abs() + 0.5
    n = torch.tensor([391], dtype=torch.int32, device="cuda")
    q[0, news - 1, group - 1, 0] = -math.inf
    account = torch.zeros(1, 1, 400, device="cuda")
    out = L.cache_attend(q, k, v, n, account)
    assert (out[0, news - 1, group - 1] == 0).all()
    q64 = q.double().cpu()
    q64[0, news - 1, group - 1] = 0.0
    want, added, _ = plain.attend(q64, k.double().cpu(), v.double().cpu(), [391], width ** -0.5)
    # that row, with a query of zeros, gave each of its 391 entries the same
    added -= 1.0 / 391
    got = account.double().cpu()[0, 0, :391]
    assert torch.isfinite(got).all()
    # logits are sums of `width` products below 8 * 4 each in fp32, weights within e^(2 delta) (as in test_gpu_cache)
    delta = (width + 4) * 2.0 ** -24 * width ** 0.5 * 32
    bound = (2 * delta + 2.0 ** -22 + news * group * 2.0 ** -23) * (added[0, 0, :391] + 1.0 / 391) + 1e-9
    assert ((got - added[0, 0, :391]).abs() <= bound).all()
