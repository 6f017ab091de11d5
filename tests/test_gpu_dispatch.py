"""Dispatch of tokens to experts and back, on the GPU, against plain 64-bit forms.

The plan and the rows that are only moved are compared exactly.  Tolerances:
a sum of k products in fp32 is within (k + 1) 2^-24 of the sum of their
sizes, one of `width` products within (width + 1) 2^-24; then half an ulp of
the output's type.
"""
import pytest

import hard_plain as plain

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_ULP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


def choices(tokens, k, experts, seed, dropped=0.0, skew=False):
    g = torch.Generator().manual_seed(seed)
    score = torch.rand(tokens, max(experts, k), generator=g)
    if skew:
        score[:, 0] += 0.9
    c = torch.argsort(score, 1, descending=True)[:, :k].int() % experts
    c[torch.rand(tokens, k, generator=g) < dropped] = -1
    return c


@pytest.mark.parametrize("tokens,k,experts", [
    (1, 1, 1), (1, 8, 256), (24, 8, 256), (63, 1, 3), (128, 8, 64), (129, 8, 64), (1000, 2, 1000), (777, 5, 60),
    (5000, 8, 256), (2048, 32, 1024), (40000, 2, 8)])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_plan(L, tokens, k, experts, dropped):
    c = choices(tokens, k, experts, tokens + k, dropped, skew=tokens % 2 == 0)
    got = L.dispatch_plan(c.cuda(), experts)
    for a, b in zip(got, plain.plan(c, experts)):
        assert torch.equal(a.cpu(), b)


def test_plan_drops_what_names_no_expert(L):
    c = torch.tensor([[0, 5, 2], [7, -1, 2], [-2 ** 31, 2 ** 31 - 1, 6]], dtype=torch.int32)
    got = L.dispatch_plan(c.cuda(), 7)
    for a, b in zip(got, plain.plan(c, 7)):
        assert torch.equal(a.cpu(), b)
    nothing = L.dispatch_plan(torch.full((1500, 2), -1, dtype=torch.int32, device="cuda"), 9)
    assert nothing[0].abs().max() == 0 and (nothing[1] == -1).all() and (nothing[2] == -1).all()


def rows(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(TYPES[dtype])


def check_all(L, tokens, k, experts, width, dtype, dropped=0.2, x=None, dy=None):
    c = choices(tokens, k, experts, tokens + width, dropped)
    offsets, slot, order = L.dispatch_plan(c.cuda(), experts)
    po, ps, _ = plain.plan(c, experts)
    there = (ps >= 0)
    at = ps.clamp(min=0).long()
    x = rows((tokens, width), 1, dtype).cuda() if x is None else x
    dy = rows((tokens, width), 2, dtype).cuda() if dy is None else dy
    ys, dxs = rows((tokens * k, width), 3, dtype), rows((tokens * k, width), 4, dtype)
    w = torch.rand(tokens, k, generator=torch.Generator().manual_seed(5)) + 0.1
    placed = int(po[-1])

    xs = L.dispatch_forward(x, slot, offsets).cpu()
    want = torch.zeros(tokens * k, width, dtype=TYPES[dtype])
    want[ps[there].long()] = x.cpu().repeat_interleave(k, 0)[there.flatten()]
    assert torch.equal(xs, want)

    def near(got, want, size, terms, ulp):
        err = (got.double().cpu() - want).abs()
        assert (err <= (terms + 1) * 2.0 ** -24 * size + ulp * want.abs() + 2.0 ** -25).all()

    y = L.combine_forward(ys.cuda(), slot, w.cuda())
    assert y.dtype == TYPES[dtype]
    terms = w.double()[:, :, None] * ys.double()[at] * there[:, :, None]
    near(y, terms.sum(1), terms.abs().sum(1), k, HALF_ULP[dtype])

    dx = L.dispatch_backward(dxs.cuda(), slot)
    terms = dxs.double()[at] * there[:, :, None]
    near(dx, terms.sum(1), terms.abs().sum(1), k, HALF_ULP[dtype])

    dys, dw = L.combine_backward(dy, ys.cuda(), slot, w.cuda(), offsets)
    d = dy.double().cpu()
    terms = ys.double()[at] * d[:, None, :] * there[:, :, None]
    near(dw, terms.sum(2), terms.abs().sum(2), width, 2.0 ** -24)
    assert (dw.cpu()[~there] == 0).all()
    want = torch.zeros(tokens * k, width, dtype=torch.float64)
    want[ps[there].long()] = (d[:, None, :] * w.double()[:, :, None]).reshape(-1, width)[there.flatten()]
    near(dys, want, want.abs(), 0, HALF_ULP[dtype])
    assert (dys[placed:] == 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("tokens,k,experts,width", [
    (1, 1, 1, 1), (3, 2, 4, 7), (17, 8, 32, 64), (50, 6, 60, 100), (33, 1, 8, 520), (20, 32, 64, 129),
    (9, 4, 16, 2048), (5, 3, 8, 2056), (4, 2, 8, 5001), (300, 2, 16, 16)])
def test_rows(L, tokens, k, experts, width, dtype):
    check_all(L, tokens, k, experts, width, dtype)


def test_rows_no_pair_and_every_pair(L):
    check_all(L, 40, 4, 8, 256, "bf16", dropped=1.1)
    check_all(L, 40, 4, 8, 256, "bf16", dropped=0.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (5, 3), (8, 8)])
def test_strided_token_rows(L, dtype, pad, shift):
    def wide(seed):
        t = torch.full((30, 256 + pad + shift), float("nan"), dtype=TYPES[dtype], device="cuda")
        t[:, shift:shift + 256] = rows((30, 256), seed, dtype).cuda()
        return t[:, shift:shift + 256]
    check_all(L, 30, 3, 8, 256, dtype, x=wide(8), dy=wide(9))
    one = rows((1, 256), 10, dtype).cuda().expand(30, 256)  # the same row for every token
    check_all(L, 30, 3, 8, 256, dtype, x=one, dy=one)


def test_dropped_pairs_and_odd_values_leave_no_trace(L):
    c = torch.tensor([[0, -1], [1, 0]], dtype=torch.int32)
    offsets, slot, _ = L.dispatch_plan(c.cuda(), 2)
    ys = torch.ones(4, 8, device="cuda")
    ys[3] = float("nan")  # behind the last pair
    w = torch.tensor([[2.0, float("nan")], [1.0, 3.0]], device="cuda")
    assert torch.equal(L.combine_forward(ys, slot, w), torch.tensor([[2.0], [4.0]], device="cuda").expand(2, 8))
    dys, dw = L.combine_backward(torch.ones(2, 8, device="cuda"), ys, slot, w, offsets)
    assert dw.tolist() == [[8.0, 0.0], [8.0, 8.0]] and dys[:, 0].tolist() == [2.0, 3.0, 1.0, 0.0]


def test_slots_out_of_range_are_ignored(L):
    ys = torch.ones(4, 8, device="cuda")
    slot = torch.tensor([[0, 4], [-5, 2 ** 30]], dtype=torch.int32, device="cuda")
    w = torch.ones(2, 2, device="cuda")
    assert L.combine_forward(ys, slot, w)[:, 0].tolist() == [1.0, 0.0]
    assert L.dispatch_backward(ys, slot)[:, 0].tolist() == [1.0, 0.0]


def test_autograd_against_differences(L):
    """The pair of dispatch and combine is linear in each argument, so differences of any size are exact."""
    g = torch.Generator().manual_seed(12)
    c = choices(6, 3, 5, 2, 0.2).cuda()
    offsets, slot, order = L.dispatch_plan(c, 5)
    x = torch.randint(-4, 5, (6, 16), generator=g).float().cuda().requires_grad_(True)
    w = (torch.randint(1, 5, (6, 3), generator=g).float() / 4).cuda().requires_grad_(True)
    up = torch.randint(-3, 4, (6, 16), generator=g).float().cuda()

    def loss(x, w):
        return (L.combine(2.0 * L.dispatch(x, slot, offsets), w, slot, offsets) * up).sum()

    loss(x, w).backward()
    with torch.no_grad():
        for i, j in ((0, 0), (3, 7), (5, 15)):
            e = torch.zeros_like(x)
            e[i, j] = 1.0
            assert float((loss(x + e, w) - loss(x - e, w)) / 2) == pytest.approx(float(x.grad[i, j]), abs=1e-3)
        for i, j in ((0, 0), (2, 1), (5, 2)):
            e = torch.zeros_like(w)
            e[i, j] = 1.0
            assert float((loss(x, w + e) - loss(x, w - e)) / 2) == pytest.approx(float(w.grad[i, j]), abs=1e-3)


def test_many_rows_pass_32_bits(L):
    """Offsets past 2^32 bytes: 40000 tokens, 3 choices, rows of 20000 elements (4.8 GB)."""
    tokens, k, width = 40000, 3, 20000
    c = choices(tokens, k, 4, 77).cuda()
    offsets, slot, order = L.dispatch_plan(c, 4)
    x = torch.arange(tokens, device="cuda").remainder(251).to(torch.bfloat16)[:, None].expand(tokens, width)
    xs = L.dispatch_forward(x.contiguous(), slot, offsets)
    assert torch.equal(xs[:, 0].long(), (order // k).remainder(251).long())
    assert torch.equal(xs[:, -1].long(), (order // k).remainder(251).long())
    dx = L.dispatch_backward(xs, slot)
    assert torch.equal(dx[:, -1].float(), (3.0 * x[:, 0].float()).to(torch.bfloat16).float())


def test_graph_and_other_stream(L):
    c = choices(3000, 4, 64, 5, 0.1).cuda()
    x = rows((3000, 256), 1, "bf16").cuda()
    w = torch.rand(3000, 4, device="cuda")
    offsets, slot, order = L.dispatch_plan(c, 64)
    y = L.combine_forward(L.dispatch_forward(x, slot, offsets), slot, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, s2, r2 = L.dispatch_plan(c, 64)
        y2 = L.combine_forward(L.dispatch_forward(x, s2, o2), s2, w)
    side.synchronize()
    assert torch.equal(order, r2) and torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    y3 = torch.empty_like(y)
    with torch.cuda.graph(graph):
        o3, s3, r3 = L.dispatch_plan(c, 64)
        L.combine_forward(L.dispatch_forward(x, s3, o3), s3, w, out=y3)
    for _ in range(3):
        y3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y3) and torch.equal(order, r3)


def test_no_tokens(L):
    offsets, slot, order = L.dispatch_plan(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 5)
    assert offsets.tolist() == [0] * 6
    xs = L.dispatch_forward(torch.empty(0, 32, device="cuda"), slot, offsets)
    assert xs.shape == (0, 32) and L.combine_forward(xs, slot, torch.empty(0, 2, device="cuda")).shape == (0, 32)


def test_refusals(L):
    c = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    offsets, slot, order = L.dispatch_plan(c, 4)
    x = torch.randn(4, 8, device="cuda")
    for bad in (lambda: L.dispatch_plan(c.cpu(), 4), lambda: L.dispatch_plan(c.long(), 4),
                lambda: L.dispatch_plan(c, 0), lambda: L.dispatch_plan(c, 1025),
                lambda: L.dispatch_forward(x.double(), slot, offsets), lambda: L.dispatch_forward(x[:3], slot, offsets),
                lambda: L.combine_forward(x, slot, torch.ones(4, 2, device="cuda")),
                lambda: L.combine_forward(torch.randn(8, 8, device="cuda"), slot, torch.ones(4, 3, device="cuda")),
                lambda: L.combine_backward(x, x.half().repeat(2, 1), slot, torch.ones(4, 2, device="cuda"), offsets),
                lambda: L.dispatch_plan(torch.zeros(4, 33, dtype=torch.int32, device="cuda"), 64)):
        with pytest.raises(L.LapsumError):
            bad()
