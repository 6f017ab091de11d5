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
