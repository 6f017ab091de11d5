"""Cache attention with accounts, and eviction, on the GPU against plain 64-bit forms.

Eviction is compared exactly.  Tolerances of the attention: a logit is a sum
of `width` products in fp32, times the scale, so it is off by at most
delta = (width + 4) 2^-24 max(scale |q|.|k|); a weight by a factor
e^(2 delta) and 2^-22 more (exponential, sums); the weights enter the second
product with 16 bits or more, so an output is within (2 delta + 2^-15) sum p |v|,
and half an ulp of its type.  The tests add 2^-24 for values near zero."""
import math

import pytest

import hard_plain as plain

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


def cache(batch, heads, capacity, width, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(batch, heads, capacity, width, generator=g).to(TYPES[dtype])
    v = torch.randn(batch, heads, capacity, width, generator=g).to(TYPES[dtype])
    return k, v


def check_attend(L, q, k, v, lengths, dtype, scale=None, kg=None, vg=None, plain_v=None):
    """kg, vg: the cache as the GPU gets it (other strides, values behind the lengths)."""
    batch, news, q_heads, width = q.shape
    scale_ = width ** -0.5 if scale is None else scale
    kg = k.cuda() if kg is None else kg
    vg = v.cuda() if vg is None else vg
    n = torch.tensor(lengths, dtype=torch.int32)
    account = torch.rand(k.shape[:3], generator=torch.Generator().manual_seed(99))
    written = torch.full(k.shape[:3], -7.0, device="cuda")
    out = L.cache_attend(q.cuda(), kg, vg, n.cuda(), account.cuda(), account_out=written, scale=scale)
    want, added, size = plain.attend(q.double(), k.double(), (v if plain_v is None else plain_v).double(), lengths, scale_)
    group = q_heads // k.shape[1]
    kk = k.double().abs().repeat_interleave(group, 1)
    reach = 0.0
    for b in range(batch):
        m = max(0, min(k.shape[2], lengths[b]))
        if m:
            reach = max(reach, float((q[b].double().abs().transpose(0, 1) @ kk[b, :, :m].transpose(1, 2)).max()))
    delta = (width + 4) * 2.0 ** -24 * reach * abs(scale_)
    err = (out.double().cpu() - want).abs()
    bound = (2 * delta + 2.0 ** -15) * size + HALF_ULP[dtype] * want.abs() + 2.0 ** -24
    assert (err <= bound).all(), float((err / bound).max())
    got = written.double().cpu()
    there = torch.arange(k.shape[2]) < n.clamp(0, k.shape[2])[:, None, None]
    there = there.expand(got.shape)
    assert (got[~there] == -7.0).all()
    terms = news * group
    err = (got - account.double() - added).abs()
    bound = (2 * delta + 2.0 ** -22 + terms * 2.0 ** -24) * added + 2.0 ** -24 * (account.double() + added) + 1e-9
    assert (err <= bound)[there].all(), float((err / bound)[there].max())
    # without accounts the output is the same
    plain_out = L.cache_attend(q.cuda(), kg, vg, n.cuda(), scale=scale)
    assert (plain_out.double().cpu() - want).abs().le((2 * delta + 2.0 ** -15) * size + HALF_ULP[dtype] * want.abs() +
                                                      2.0 ** -24).all()
    return out


def query(batch, news, heads, width, dtype, seed=1, gain=2.0):
    return (gain * torch.randn(batch, news, heads, width, generator=torch.Generator().manual_seed(seed))).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("width", [8, 24, 64, 72, 80, 96, 120, 128, 136, 192, 256])
def test_widths(L, width, dtype):
    k, v = cache(2, 2, 150, width, dtype)
    for news, group in ((1, 4), (3, 7)):
        check_attend(L, query(2, news, 2 * group, width, dtype), k, v, [150, 77], dtype)


@pytest.mark.parametrize("heads,group,news", [
    (1, 1, 1), (3, 1, 1), (2, 8, 1), (1, 16, 1), (1, 17, 1), (2, 5, 3), (1, 1, 16), (1, 8, 4), (1, 4, 33), (1, 32, 5),
    (2, 1, 70)])
def test_head_layouts(L, heads, group, news):
    k, v = cache(2, heads, 300, 64, "bf16", seed=heads + group)
    check_attend(L, query(2, news, heads * group, 64, "bf16"), k, v, [300, 131], "bf16")


@pytest.mark.parametrize("news,group", [(1, 4), (5, 4), (20, 2)])
@pytest.mark.parametrize("capacity", [1, 2, 31, 32, 33, 127, 128, 129, 256, 1000, 3001])
def test_lengths(L, capacity, news, group):
    lengths = sorted({0, 1, capacity // 2, capacity - 1, capacity})
    k, v = cache(len(lengths), 1, capacity, 64, "bf16", seed=capacity)
    check_attend(L, query(len(lengths), news, group, 64, "bf16"), k, v, lengths, "bf16")


def test_lengths_out_of_range_are_clamped(L):
    k, v = cache(3, 1, 100, 64, "fp16")
    check_attend(L, query(3, 1, 2, 64, "fp16"), k, v, [-5, 101, 2 ** 31 - 1], "fp16")


@pytest.mark.parametrize("width,dtype", [(128, "bf16"), (64, "fp16"), (256, "bf16")])
def test_long(L, width, dtype):
    k, v = cache(1, 1, 20011, width, dtype, seed=3)
    check_attend(L, query(1, 1, 8, width, dtype), k, v, [20003], dtype)
    check_attend(L, query(1, 12, 3, width, dtype), k, v, [20011], dtype)


def test_scale_and_sharp_weights(L):
    k, v = cache(1, 2, 400, 128, "bf16", seed=4)
    q = query(1, 2, 4, 128, "bf16")
    for scale in (0.0, 1.0, -0.3, 0.01):
        check_attend(L, q, k, v, [399], "bf16", scale=scale)


@pytest.mark.parametrize("batch,news,capacity", [(1, 1, 200), (256, 40, 1024), (256, 1, 1000), (64, 20, 5000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_light_entries_beside_a_heavy_one(L, dtype, batch, news, capacity):
    """Entry 0 outweighs each other one 1.2e7 times and its value is 0: the output is what the others weigh together.
    A weight's part in the products is within 2^-32 of the heaviest's, or 2^-16 of itself, and the output is rounded."""
    z = 16.296875
    k = torch.zeros(batch, 1, capacity, 64, dtype=TYPES[dtype], device="cuda")
    v = torch.ones_like(k)
    k[:, :, 0, 0], v[:, :, 0] = 4.0, 0.0
    q = torch.zeros(batch, news, 1, 64, dtype=TYPES[dtype], device="cuda")
    q[:, :, 0, 0] = z / 4  # a bf16 number is not needed: the logit below is that of the rounded one
    p = math.exp(-4.0 * float(q[0, 0, 0, 0]))
    others = torch.arange(capacity - news, capacity).double() * p
    want = (others / (1.0 + others))[None, :, None, None]
    n = torch.full((batch,), capacity, dtype=torch.int32, device="cuda")
    account = torch.zeros(batch, 1, capacity, device="cuda")
    out = L.cache_attend(q, k, v, n, account, scale=1.0).double().cpu()
    bound = 2.0 ** -32 / p + 2.0 ** -16 + HALF_ULP[dtype] + 2.0 ** -18
    assert ((out - want).abs() <= bound * want + 2.0 ** -25).all()
    got = account[:, 0, 1].double().cpu() / news  # entry 1 is seen by every token
    assert ((got / (p / (1.0 + others)).mean() - 1.0).abs() <= 2.0 ** -18).all()


def test_many_caches(L):
    k, v = cache(40, 8, 64, 64, "bf16", seed=5)
    check_attend(L, query(40, 1, 16, 64, "bf16"), k, v, [int(x) for x in torch.arange(40) + 20], "bf16")


@pytest.mark.parametrize("news,group", [(1, 4), (6, 3), (9, 4)])
@pytest.mark.parametrize("odd", [math.nan, math.inf, -math.inf])
def test_what_a_token_does_not_see_does_not_reach_it(L, news, group, odd):
    """Values behind the lengths, and for every token the newer tokens' values and keys, may be anything."""
    lengths = [200, 45, 3]
    k, v = cache(3, 2, 210, 64, "bf16", seed=6)
    q = query(3, news, 2 * group, 64, "bf16")
    kg, vg = k.clone(), v.clone()
    for b, n in enumerate(lengths):
        kg[b, :, n:] = odd
        vg[b, :, n:] = odd
    check_attend(L, q, k, v, lengths, "bf16", kg=kg.cuda(), vg=vg.cuda())
    if news == 1:
        return
    for b, n in enumerate(lengths):  # the newest token's own value is seen by that token alone
        vg[b, :, n - 1, ::3] = odd
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    out = L.cache_attend(q.cuda(), kg.cuda(), vg.cuda(), n)
    clean = L.cache_attend(q.cuda(), kg.cuda(), v.cuda(), n)
    assert torch.equal(out[:2, :-1], clean[:2, :-1])
    assert torch.equal(out[2, :-1], clean[2, :-1])
    assert not torch.isfinite(out[:, -1, :, 0]).any() and torch.equal(out[:, -1, :, 1], clean[:, -1, :, 1])


def test_strided_caches(L):
    """Entry-major storage, a slice of a longer cache, and heads shared by all sequences."""
    k, v = cache(2, 3, 90, 64, "bf16", seed=7)
    q = query(2, 2, 6, 64, "bf16")
    major = [x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for x in (k, v)]
    a = check_attend(L, q, k, v, [90, 50], "bf16", kg=major[0], vg=major[1])
    longer = [torch.full((2, 3, 200, 80), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, x in zip(longer, (k, v)):
        t[:, :, 50:140, 8:72] = x.cuda()
    b = check_attend(L, q, k, v, [90, 50], "bf16", kg=longer[0][:, :, 50:140, 8:72], vg=longer[1][:, :, 50:140, 8:72])
    assert torch.equal(a, b)
    one = [x[:1].cuda().expand(2, 3, 90, 64) for x in (k, v)]
    check_attend(L, q, k[:1].expand(2, 3, 90, 64), v[:1].expand(2, 3, 90, 64), [90, 50], "bf16", kg=one[0], vg=one[1])


def test_offsets_past_32_bits(L):
    """A cache of 8.6 GB per tensor: its last sequence lies past 2^32 bytes."""
    k = torch.zeros(2, 1, 16_800_000, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[1, 0, 16_799_990, :] = 4.0
    v[1, 0, 16_799_990, :] = torch.arange(128, device="cuda").bfloat16()
    q = torch.ones(2, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([5, 16_800_000], dtype=torch.int32, device="cuda")
    account = torch.zeros(2, 1, 16_800_000, device="cuda")
    out = L.cache_attend(q, k, v, n, account)
    # logits 45.25 and 0: weight 1 / (1 + 16.8e6 e^-45.25) = 1 - 4e-13
    assert torch.equal(out[1, 0], v[1, :, 16_799_990].expand(4, 128))
    assert out[0].abs().max() == 0 and float(account[1, 0, 16_799_990]) == pytest.approx(4.0, abs=1e-6)
    assert account[0, 0, :5].tolist() == pytest.approx([0.8] * 5, abs=1e-6) and account[0, 0, 5:].abs().max() == 0
    del k, v, account


def test_accounts_in_place_graph_and_other_stream(L):
    k, v = (x.cuda() for x in cache(3, 2, 500, 128, "bf16", seed=8))
    q = query(3, 1, 8, 128, "bf16").cuda()
    n = torch.tensor([500, 17, 333], dtype=torch.int32, device="cuda")
    account = torch.rand(3, 2, 500, device="cuda")
    apart = torch.zeros_like(account)
    out = L.cache_attend(q, k, v, n, account, account_out=apart)
    side = torch.cuda.Stream()
    here = account.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2 = L.cache_attend(q, k, v, n, here)
    side.synchronize()
    assert torch.equal(out, out2)
    for b, m in enumerate(n.tolist()):
        assert torch.equal(here[b, :, :m], apart[b, :, :m]) and torch.equal(here[b, :, m:], account[b, :, m:])
    graph = torch.cuda.CUDAGraph()
    out3, apart3 = torch.empty_like(out), torch.zeros_like(account)
    with torch.cuda.graph(graph):
        L.cache_attend(q, k, v, n, account, account_out=apart3, out=out3)
    for _ in range(3):
        out3.zero_(), apart3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out3) and torch.equal(apart, apart3)


def test_attend_refusals(L):
    k, v = (x.cuda() for x in cache(2, 2, 20, 64, "bf16"))
    q = query(2, 1, 4, 64, "bf16").cuda()
    n = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    acc = torch.zeros(2, 2, 20, device="cuda")
    for bad in (lambda: L.cache_attend(q.cpu(), k, v, n), lambda: L.cache_attend(q.half(), k, v, n),
                lambda: L.cache_attend(q.float(), k.float(), v.float(), n), lambda: L.cache_attend(q, k, v[:, :1], n),
                lambda: L.cache_attend(q[:, :, :3], k, v, n), lambda: L.cache_attend(q, k, v, n.long()),
                lambda: L.cache_attend(q, k, v, n, acc[:, :1]), lambda: L.cache_attend(q, k, v, n, account_out=acc),
                lambda: L.cache_attend(q, k, v, n, scale=math.inf),
                lambda: L.cache_attend(q[..., :60], k[..., :60], v[..., :60], n),
                lambda: L.cache_attend(q[..., :56], k[..., 4:60], v[..., 4:60], n),
                lambda: L.cache_attend(q, k, v, n, acc.transpose(0, 1)),
                lambda: L.cache_attend(q[..., ::2], k[..., ::2], v[..., ::2], n)):
        with pytest.raises(L.LapsumError):
            bad()


# --------------------------------------------------------------- eviction
def check_evict(L, batch, heads, capacity, width, lengths, keep, accounts=None, positions=None, sinks=0, recent=0,
                next_position=None, in_place=False, dtype="bf16", major=False):
    g = torch.Generator().manual_seed(capacity + keep)
    k, v = cache(batch, heads, capacity, width, dtype, seed=keep)
    if accounts is None:
        accounts = torch.rand(batch, heads, capacity, generator=g)
    if positions is None:
        positions = torch.argsort(torch.rand(batch, heads, capacity, generator=g), 2).int()
    if next_position is None:
        next_position = [capacity] * batch
    kept, after = plain.evict(accounts, positions, lengths, keep, next_position, sinks, recent)
    kg, vg = k.cuda(), v.cuda()
    if major:
        kg, vg = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (kg, vg))
    ag, pg = accounts.cuda(), positions.cuda()
    ao = ag if in_place else torch.full_like(ag, -3.0)
    po = pg if in_place else torch.full_like(pg, -3)
    got, n = L.cache_evict(kg, vg, ag, pg, torch.tensor(lengths, dtype=torch.int32).cuda(), keep,
                           next_position=torch.tensor(next_position, dtype=torch.int32).cuda(), sinks=sinks,
                           recent=recent, account_out=None if in_place else ao, positions_out=None if in_place else po)
    assert torch.equal(n.cpu(), after) and torch.equal(got.cpu(), kept)
    for b in range(batch):
        m = int(after[b])
        for h in range(heads):
            src = kept[b, h, :m].long()
            for now, before in ((kg, k), (vg, v)):
                assert torch.equal(now[b, h, :m].cpu(), before[b, h][src])
                assert torch.equal(now[b, h, m:].cpu(), before[b, h, m:])
            assert torch.equal(ao[b, h, :m].cpu().nan_to_num(nan=-1e30), accounts[b, h][src].nan_to_num(nan=-1e30))
            assert torch.equal(po[b, h, :m].cpu(), positions[b, h][src])
            if not in_place:
                assert (ao[b, h, m:] == -3.0).all() and (po[b, h, m:] == -3).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("capacity,lengths,keep", [
    (1, [1, 0], 1), (2, [2, 1], 1), (65, [65, 64], 64), (100, [100, 40], 10), (100, [99, 51], 50), (300, [300, 0], 1),
    (1023, [1023, 1000], 1000), (1024, [1024, 1025], 1023), (1025, [1025, 3], 1024), (4097, [4097, 4096], 4096),
    (2500, [2500, 2049], 2048), (2500, [2477, 2100], 1111), (5000, [4999, 1], 2), (5000, [-4, 9999], 300),
    (10000, [10000, 9999], 2500), (9001, [8999, 8200], 8192)])
def test_evict_lengths(L, capacity, lengths, keep, in_place):
    check_evict(L, 2, 2, capacity, 64, lengths, keep, in_place=in_place)


@pytest.mark.parametrize("width", [8, 40, 96, 128, 200, 256])
def test_evict_widths(L, width):
    check_evict(L, 2, 1, 400, width, [400, 350], 200, dtype="fp16")
    check_evict(L, 1, 3, 400, width, [333], 100, major=True)


@pytest.mark.parametrize("sinks,recent", [(4, 0), (0, 16), (4, 30), (60, 60), (0, 1000)])
@pytest.mark.parametrize("keep", [20, 64, 119])
def test_evict_protected(L, sinks, recent, keep):
    check_evict(L, 2, 2, 120, 64, [120, 110], keep, sinks=sinks, recent=recent, next_position=[120, 115])


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "nan", "infinite", "signs", "digits"])
@pytest.mark.parametrize("capacity,keep", [(200, 60), (3000, 2999), (3000, 1500), (20000, 5000)])
def test_evict_accounts(L, kind, capacity, keep):
    g = torch.Generator().manual_seed(5)
    a = torch.rand(1, 2, capacity, generator=g)
    if kind == "equal":
        a[:] = 0.25
    elif kind == "zeros":
        a[a < 0.7] = 0.0
        a[0, 0, ::7] = -0.0
    elif kind == "few":
        a = (a * 4).floor() / 4
    elif kind == "nan":
        a[a < 0.6] = math.nan
        a[0, 1] = math.nan
    elif kind == "infinite":
        a[a < 0.3] = -math.inf
        a[a > 0.8] = math.inf
    elif kind == "signs":
        a = a - 0.5
    else:  # keys that differ in their last bits only
        a = 1.0 + torch.randint(0, 300, a.shape, generator=g) * 2.0 ** -23
    check_evict(L, 1, 2, capacity, 16, [capacity], keep, accounts=a, sinks=2)


def test_evict_long_row(L):
    """131072 entries to a quarter, and one over the budget, against a sort."""
    g = torch.Generator().manual_seed(6)
    for lengths, keep, kind in (([130001, 131072], 32768, ""), ([131072, 131000], 131071, ""),
                                ([131072, 70000], 65536, "few"), ([100000, 20], 4096, "equal"),
                                ([131072, 131072], 9, "few"), ([131072, 4097], 4096, "")):
        s = 131072
        a = torch.exp(2 * torch.randn(2, 1, s, generator=g)).cuda()
        if kind == "few":
            a = a.ceil().clamp(max=5.0)
        elif kind == "equal":
            a[:] = 1.0
        p = torch.arange(s, dtype=torch.int32).expand(2, 1, s).contiguous().cuda()
        k, v = (x.cuda() for x in cache(2, 1, s, 16, "bf16", seed=9))
        k0, v0 = k.clone(), v.clone()
        n = torch.tensor(lengths, dtype=torch.int32).cuda()
        kept, after = L.cache_evict(k, v, a, p, n, keep, account_out=torch.empty_like(a),
                                    positions_out=torch.empty_like(p))
        for b in range(2):
            m = min(lengths[b], keep)
            top = torch.sort(a[b, 0, :lengths[b]], descending=True, stable=True).indices[:m]
            got = kept[b, 0, :m].long()
            assert torch.equal(torch.sort(got).values, torch.sort(top).values)
            stay = got[got < m]
            assert torch.equal(stay, torch.nonzero(got < m)[:, 0]) and (kept[b, 0, m:] == -1).all()
            moved = got[got >= m]
            assert torch.equal(moved, torch.sort(moved).values)
            assert torch.equal(k[b, 0, :m], k0[b, 0][got]) and torch.equal(v[b, 0, :m], v0[b, 0][got])


def test_evict_many_rows(L):
    check_evict(L, 33, 8, 70, 16, [70 - i for i in range(33)], 41, sinks=1, recent=4, next_position=[90] * 33)


def test_evict_graph_and_other_stream(L):
    k, v = (x.cuda() for x in cache(2, 2, 3000, 64, "bf16", seed=10))
    a = torch.rand(2, 2, 3000, device="cuda")
    p = torch.arange(3000, dtype=torch.int32, device="cuda").expand(2, 2, 3000).contiguous()
    n = torch.tensor([3000, 2500], dtype=torch.int32, device="cuda")
    k1, v1 = k.clone(), v.clone()
    a1, p1 = torch.zeros_like(a), torch.zeros_like(p)
    kept, after = L.cache_evict(k1, v1, a, p, n, 1000, account_out=a1, positions_out=p1)
    side = torch.cuda.Stream()
    k2, v2 = k.clone(), v.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kept2, _ = L.cache_evict(k2, v2, a, p, n, 1000, account_out=torch.zeros_like(a), positions_out=torch.zeros_like(p))
    side.synchronize()
    assert torch.equal(kept, kept2) and torch.equal(k1, k2) and torch.equal(v1, v2)
    graph = torch.cuda.CUDAGraph()
    k3, v3 = k.clone(), v.clone()
    a3, p3 = torch.zeros_like(a), torch.zeros_like(p)
    with torch.cuda.graph(graph):
        kept3, after3 = L.cache_evict(k3, v3, a, p, n, 1000, account_out=a3, positions_out=p3)
    for _ in range(3):
        k3.copy_(k), v3.copy_(v), a3.zero_(), p3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, kept3) and torch.equal(k1, k3) and torch.equal(a1, a3) and torch.equal(p1, p3)


def test_evict_refusals(L):
    k, v = (x.cuda() for x in cache(2, 2, 20, 64, "bf16"))
    a = torch.zeros(2, 2, 20, device="cuda")
    p = torch.zeros(2, 2, 20, dtype=torch.int32, device="cuda")
    n = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    for bad in (lambda: L.cache_evict(k.cpu(), v, a, p, n, 5), lambda: L.cache_evict(k, v, a.double(), p, n, 5),
                lambda: L.cache_evict(k, v, a, p.long(), n, 5), lambda: L.cache_evict(k, v, a, p, n, 0),
                lambda: L.cache_evict(k, v, a, p, n, 21), lambda: L.cache_evict(k, v, a, p, n, 5, recent=3),
                lambda: L.cache_evict(k, v, a, p, n, 5, sinks=-1), lambda: L.cache_evict(k, v, a, p, n, 5, recent=-1),
                lambda: L.cache_evict(k[:, :1].expand(2, 2, 20, 64), v, a, p, n, 5),
                lambda: L.cache_evict(k, v, a.transpose(0, 1), p, n, 5),
                lambda: L.cache_evict(k.float(), v.float(), a, p, n, 5)):
        with pytest.raises(L.LapsumError):
            bad()


@pytest.mark.parametrize("news,group,width", [(1, 4, 64), (1, 16, 128), (3, 2, 96), (1, 1, 256), (2, 5, 64)])
@pytest.mark.parametrize("capacity", [1, 31, 256, 700, 1500])
def test_many_short_caches(L, capacity, news, group, width):
    """260 caches: each is finished by one workgroup where its logits fit, with and without accounts."""
    lengths = [max(0, capacity - 3 * i) for i in range(130)]
    k, v = cache(130, 2, capacity, width, "bf16", seed=capacity + width)
    few = [0, 1, 7, 129]
    q = query(130, news, 2 * group, width, "bf16")
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    account = torch.rand(130, 2, capacity, device="cuda")
    apart = torch.full_like(account, -7.0)
    out = L.cache_attend(q.cuda(), k.cuda(), v.cuda(), n, account, account_out=apart)
    # the same sequences by themselves (checked against the plain form), whatever their number chose
    pick = torch.tensor(few)
    alone = check_attend(L, q[pick], k[pick], v[pick], [lengths[i] for i in few], "bf16")
    assert (out[pick.cuda()].float() - alone.float()).abs().max() <= 2.0 ** -7 * (1 + alone.float().abs().max())
    check_attend(L, q[:3].repeat(44, 1, 1, 1)[:130], k[:3].repeat(44, 1, 1, 1)[:130], v[:3].repeat(44, 1, 1, 1)[:130],
                 [lengths[i % 3] for i in range(130)], "bf16") if capacity <= 31 else None
    for b in few:
        m = lengths[b]
        want = plain.attend(q[b:b + 1].double(), k[b:b + 1].double(), v[b:b + 1].double(), [m], width ** -0.5)[1]
        got = apart[b].double().cpu() - account[b].double().cpu()
        assert (got[:, :m] - want[0, :, :m]).abs().max() <= 1e-5 * news * group if m else True
        assert (apart[b, :, m:] == -7.0).all()
