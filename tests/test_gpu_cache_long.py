"""The cache operators over what the short cases do not reach: many new tokens (a prompt, or a part of one), caches
whose capacity is far above what they hold, wide entries in caches that one workgroup takes whole, and evictions of
long rows in place, at every width, with protected entries, and past the tiles that a workgroup preloads.

Attention's tolerances are those of test_gpu_cache; evictions are compared exactly."""
import math

import numpy as np
import pytest

import hard_plain as plain
import test_gpu_cache as c

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


# ------------------------------------------------------- many new tokens
@pytest.mark.parametrize("news,group,width,capacity,lengths", [
    (130, 2, 64, 130, [130, 129]),        # prompts as long as their caches, and one token short of it
    (200, 1, 128, 700, [650, 200, 7]),    # parts of prompts, one longer than what is there
    (257, 3, 96, 300, [300]),
    (512, 1, 64, 512, [512]),
    (512, 1, 128, 2000, [1999]),
    (90, 4, 256, 400, [400, 90]),
    (1000, 1, 24, 1000, [1000])])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_new_tokens(L, news, group, width, capacity, lengths, dtype):
    k, v = c.cache(len(lengths), 1, capacity, width, dtype, seed=news)
    c.check_attend(L, c.query(len(lengths), news, group, width, dtype), k, v, lengths, dtype)


def test_many_new_tokens_see_no_newer_one(L):
    """Values and keys of newer tokens may be anything to the older ones, over several blocks."""
    k, v = (x.cuda() for x in c.cache(1, 1, 400, 64, "bf16", seed=3))
    q = c.query(1, 150, 2, 64, "bf16").cuda()
    n = torch.tensor([400], dtype=torch.int32, device="cuda")
    clean = L.cache_attend(q, k, v, n)
    for at in (260, 333, 399):  # the token of entry `at` is the (at - 250)-th new one
        k2, v2 = k.clone(), v.clone()
        k2[0, 0, at], v2[0, 0, at] = math.inf, math.nan
        out = L.cache_attend(q, k2, v2, n)
        first = at - 250
        assert torch.isnan(out[:, first:]).all()
        # rows of a tile share the steps at which their bases move, so bits may change: twice the bound of
        # test_gpu_cache, with logits below 16 (delta 7e-5) and a mean |v| below 1.5
        off = (out[:, :first].float() - clean[:, :first].float()).abs()
        assert (off <= 2.0 ** -10 + 2.0 ** -7 * clean[:, :first].float().abs()).all()


# --------------------------------------------- capacity far above length
@pytest.mark.parametrize("news,group", [(1, 4), (5, 3), (20, 2), (60, 2)])
@pytest.mark.parametrize("capacity", [5000, 50000, 131072])
def test_long_caches_hold_little(L, capacity, news, group):
    lengths = [1000, 3, 0, 129]
    k, v = c.cache(4, 1, 1000, 64, "bf16", seed=capacity)
    q = c.query(4, news, group, 64, "bf16")
    account = torch.rand(4, 1, 1000, generator=torch.Generator().manual_seed(99))
    want = c.check_attend(L, q, k, v, lengths, "bf16")
    wide = [torch.full((4, 1, capacity, 64), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, x in zip(wide, (k, v)):
        t[:, :, :1000] = x.cuda()
    long = torch.full((4, 1, capacity), math.nan, device="cuda")
    long[:, :, :1000] = account.cuda()
    to = torch.full_like(long, -7.0)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = L.cache_attend(q.cuda(), wide[0], wide[1], n, long, account_out=to)
    short = torch.full((4, 1, 1000), -7.0, device="cuda")
    L.cache_attend(q.cuda(), k.cuda(), v.cuda(), n, account.cuda(), account_out=short)
    # both are within the bound of the 64-bit form (logits below 16: delta 7e-5; a mean |v| below 1.5): twice that
    assert ((out.float() - want.float()).abs() <= 2.0 ** -10 + 2.0 ** -7 * want.float().abs()).all()
    there = torch.arange(1000, device="cuda").expand(4, 1, 1000) < n[:, None, None]
    off = (to[:, :, :1000] - short).abs()
    assert (off <= 2.0 ** -11 * (1.0 + short.abs()))[there].all()
    assert (to[:, :, :1000][~there] == -7.0).all() and (to[:, :, 1000:] == -7.0).all()


@pytest.mark.parametrize("keep", [40, 999, 1000, 1500, 30000])
def test_long_caches_evict_little(L, keep):
    check_long(L, 40000, [1000, 41, 0, 39999], keep, 24)


# -------------------------------------------------- wide caches in whole
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("news,group", [(1, 4), (2, 2)])
def test_wide_whole_caches(L, news, group, dtype):
    """260 caches of 4000 entries of 256 elements, 4 rows each: logits of 64 KB beside 67 KB of outputs."""
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(130, 2, 4000, 256, generator=g, device="cuda", dtype=c.TYPES[dtype]) for _ in range(2))
    q = c.query(130, news, 2 * group, 256, dtype).cuda()
    lengths = [4000 - 13 * i for i in range(130)]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    account = torch.rand(130, 2, 4000, generator=g, device="cuda")
    to = torch.full_like(account, -7.0)
    out = L.cache_attend(q, k, v, n, account, account_out=to)
    assert (to[torch.arange(4000, device="cuda").expand(130, 2, 4000) >= n[:, None, None]] == -7.0).all()
    for b in (0, 64, 129):
        m = lengths[b]
        want, added, size = plain.attend(q[b:b + 1].double().cpu(), k[b:b + 1].double().cpu(), v[b:b + 1].double().cpu(),
                                         [m], 1 / 16)
        # logits: sums of 256 products; |q| |k| is at most 256 * 9 * 5 here, times the scale (as in test_gpu_cache)
        reach = float((q[b].double().abs().transpose(0, 1).cpu() @
                       k[b].double().abs().cpu().repeat_interleave(group, 0).transpose(1, 2)).max()) / 16
        delta = 260 * 2.0 ** -24 * reach
        err = (out[b:b + 1].double().cpu() - want).abs()
        assert (err <= (2 * delta + 2.0 ** -15) * size + c.HALF_ULP[dtype] * want.abs() + 2.0 ** -24).all()
        err = (to[b, :, :m].double().cpu() - account[b, :, :m].double().cpu() - added[0, :, :m]).abs()
        bound = (2 * delta + 2.0 ** -22 + 4 * 2.0 ** -24) * added[0, :, :m] + 2.0 ** -24 * (1.0 + added[0, :, :m]) + 1e-9
        assert (err <= bound).all()


# ---------------------------------------------------------- long evictions
def survivors(account, position, n, keep, sinks, recent, next_position):
    """kept of one row by a sort: protected entries, then by account (NaN last), then by slot."""
    m = min(n, keep)
    a, p = account[:n].astype(np.float64), position[:n].astype(np.int64)
    safe = (p < sinks) | ((p >= next_position - recent) if recent > 0 else False)
    nan = np.isnan(a) & ~safe
    rank = np.where(safe | nan, 0.0, -a)
    stays = np.sort(np.lexsort((np.arange(n), rank, nan, ~safe))[:m])
    kept = np.full(keep, -1, dtype=np.int64)
    kept[:m] = np.arange(m)
    front = stays[stays < m]
    kept[np.setdiff1d(np.arange(m), front)] = stays[stays >= m]
    return kept


def check_long(L, capacity, lengths, keep, width, sinks=0, recent=0, in_place=False, kind="", dtype="bf16"):
    batch, heads = len(lengths), 1
    g = torch.Generator(device="cuda").manual_seed(capacity + keep + width)
    k, v = (torch.randint(-2 ** 15, 2 ** 15, (batch, heads, capacity, width), generator=g, device="cuda",
                          dtype=torch.int16) for _ in range(2))  # any bits: entries are only moved
    a = torch.rand(batch, heads, capacity, generator=g, device="cuda")
    if kind == "few":
        a = (a * 5).floor()
    elif kind == "nan":
        a[a < 0.5] = math.nan
    p = torch.argsort(torch.rand(batch, heads, capacity, generator=g, device="cuda"), 2).int()
    nexts = [capacity - 3] * batch
    k1, v1, a1, p1 = k.clone(), v.clone(), a.clone(), p.clone()
    if not in_place:
        a1.fill_(-3.0), p1.fill_(-3)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kept, after = L.cache_evict(k1.view(c.TYPES[dtype]), v1.view(c.TYPES[dtype]), a1 if in_place else a,
                                p1 if in_place else p, n, keep,
                                next_position=torch.tensor(nexts, dtype=torch.int32, device="cuda"), sinks=sinks,
                                recent=recent, account_out=None if in_place else a1,
                                positions_out=None if in_place else p1)
    for b, length in enumerate(lengths):
        m = min(length, keep)
        want = torch.from_numpy(survivors(a[b, 0].cpu().numpy(), p[b, 0].cpu().numpy(), length, keep, sinks, recent,
                                          nexts[b])).cuda()
        assert int(after[b]) == m and torch.equal(kept[b, 0].long(), want)
        src = want[:m]
        for now, was in ((k1, k), (v1, v), (p1, p), (a1.view(torch.int32), a.view(torch.int32))):
            assert torch.equal(now[b, 0, :m], was[b, 0][src])
        for now, was in ((k1, k), (v1, v)):
            assert torch.equal(now[b, 0, m:], was[b, 0, m:])
        if in_place:
            assert torch.equal(p1[b, 0, m:], p[b, 0, m:])
            assert torch.equal(a1[b, 0, m:].view(torch.int32), a[b, 0, m:].view(torch.int32))
        else:
            assert (a1[b, 0, m:] == -3.0).all() and (p1[b, 0, m:] == -3).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("width", [8, 40, 96, 128, 200, 256])
@pytest.mark.parametrize("keep", [300, 9000, 19990])
def test_long_rows_at_every_width(L, width, keep, in_place):
    check_long(L, 20000, [20000, 19991], keep, width, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("sinks,recent", [(4, 0), (0, 64), (4, 512), (3000, 9000), (0, 40000)])
@pytest.mark.parametrize("kind", ["", "few", "nan"])
def test_long_rows_with_protected_entries(L, kind, sinks, recent, in_place):
    check_long(L, 33000, [33000, 32001, 20000], 8000, 16, sinks, recent, in_place, kind)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep", [600001, 1200000, 1000])
@pytest.mark.parametrize("kind", ["", "few"])
def test_rows_past_the_preloaded_tiles(L, kind, keep, in_place):
    """1200003 entries: tiles of more than the 4096 that a workgroup asks for ahead."""
    check_long(L, 1200003, [1200003], keep, 8, 4, 512, in_place, kind)
