"""The experts' products and their gradients on the GPU against their definition in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import search_plain as plain  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


def inputs(rows, n, m, offsets, dtype, stored="in_out", seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    e = len(offsets) - 1
    xs, dys = torch.randn(rows, n, generator=g).to(dt).cuda(), torch.randn(rows, m, generator=g).to(dt).cuda()
    w = torch.randn(e, n, m, generator=g).to(dt).cuda()
    if stored == "out_in":
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    return xs, w, torch.tensor(offsets, dtype=torch.int32, device="cuda"), dys


def check(L, xs, w, offsets, dys):
    ys, dxs, dw = plain.products(xs, w, offsets, dys)
    got = L.expert_product_forward(xs, w, offsets)
    assert got.dtype == xs.dtype and got.is_contiguous()
    plain.check_product(got, ys, "ys")
    dx, d = L.expert_product_backward(dys, xs, w, offsets)
    assert dx.dtype == xs.dtype and d.dtype == w.dtype and d.shape == w.shape
    plain.check_product(dx, dxs, "dxs")
    plain.check_product(d, dw, "dw")
    return got, dx, d


# rows of the experts: none, one, a few, some past a tile
RAGGED = [0, 1, 0, 33, 7, 130, 64, 0, 16]


def offsets_of(sizes, first=0):
    out = [first]
    for s in sizes:
        out.append(out[-1] + s)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("stored", ["in_out", "out_in"])
@pytest.mark.parametrize("n,m", [(64, 64), (128, 256), (264, 136), (8, 512), (520, 8), (72, 1032)])
def test_ragged(L, n, m, stored, dtype):
    offsets = offsets_of(RAGGED)
    check(L, *inputs(offsets[-1], n, m, offsets, dtype, stored))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("stored", ["in_out", "out_in"])
@pytest.mark.parametrize("n,m", [(1, 1), (1, 70), (33, 1), (7, 13), (65, 127), (100, 36), (131, 260)])
def test_sizes_of_no_whole_16_bytes(L, n, m, stored, dtype):
    offsets = offsets_of(RAGGED)
    check(L, *inputs(offsets[-1], n, m, offsets, dtype, stored))


@pytest.mark.parametrize("stored", ["in_out", "out_in"])
@pytest.mark.parametrize("rows", [1, 2, 8, 15, 16, 17, 31, 63, 64, 65, 129])
def test_one_expert(L, rows, stored):
    check(L, *inputs(rows, 96, 160, [0, rows], "bf16", stored))


@pytest.mark.parametrize("experts", [1, 2, 62, 63, 64, 255, 256, 1024])
def test_many_experts(L, experts):
    g = torch.Generator().manual_seed(experts)
    sizes = torch.randint(0, 4, (experts,), generator=g).tolist()
    sizes[0] += 1
    offsets = offsets_of(sizes)
    check(L, *inputs(offsets[-1], 64, 72, offsets, "bf16"))


@pytest.mark.parametrize("stored", ["in_out", "out_in"])
@pytest.mark.parametrize("sizes", [[300, 900, 0, 511], [257, 1, 1023, 5], [2048]])
@pytest.mark.parametrize("n,m", [(512, 768), (1032, 264)])
def test_many_rows(L, sizes, n, m, stored):
    offsets = offsets_of(sizes)
    check(L, *inputs(offsets[-1], n, m, offsets, "fp16", stored))


def check_sample(L, xs, w, offsets, dys, experts):
    """As check, for all rows of some experts: larger products than the CPU forms in time."""
    got, bounds = L.expert_product_forward(xs, w, offsets), offsets.tolist()
    dx, d = L.expert_product_backward(dys, xs, w, offsets)
    for e in experts:
        mine = slice(bounds[e], bounds[e + 1])
        if mine.start == mine.stop:
            assert (d[e] == 0).all()
            continue
        x, m, dy = xs[mine].double(), w[e].double(), dys[mine].double()
        longest = max(1, mine.stop - mine.start)
        for a, b, size, terms in ((got[mine], x @ m, x.abs() @ m.abs(), x.shape[1]),
                                  (dx[mine], dy @ m.t(), dy.abs() @ m.t().abs(), dy.shape[1]),
                                  (d[e], x.t() @ dy, x.t().abs() @ dy.abs(), longest)):
            plain.check_product(a, (b.cpu(), size.cpu(), terms), f"expert {e}")


@pytest.mark.parametrize("stored", ["in_out", "out_in"])
def test_tiles_of_every_kind(L, stored):
    """Sizes that go to each of the kernels: few rows of few and of many experts, some rows, tiles of 128 and of 256 rows; in
    each the sum is no whole number of steps, and neither rows nor columns are of tiles."""
    for experts, rows, n, m in ((3, 5, 200, 520), (200, 230, 200, 2056), (4, 300, 1032, 2056), (40, 2500, 1032, 1032),
                                (70, 33000, 264, 1288), (5, 9000, 776, 1544)):
        g = torch.Generator().manual_seed(rows)
        p = torch.softmax(0.7 * torch.randn(experts, generator=g), 0)
        sizes = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=experts).tolist()
        check_sample(L, *inputs(rows, n, m, offsets_of(sizes), "bf16", stored),
                     sorted({0, 1, experts // 2, experts - 1, sizes.index(max(sizes)), sizes.index(min(sizes))}))


@pytest.mark.parametrize("n,m", [(128, 256), (37, 50)])
def test_rows_of_no_expert_are_zero(L, n, m):
    """Rows before the first expert's and behind the last one's (another device's, or dropped pairs): NaN there stays
    there."""
    xs, w, offsets, dys = inputs(200, n, m, [40, 90, 90, 131], "bf16")
    for x in (xs, dys):
        x[:40] = float("nan")
        x[131:] = float("inf")
    clean = xs.nan_to_num(0, 0, 0), dys.nan_to_num(0, 0, 0)
    ys, dxs, dw = plain.products(clean[0], w, offsets, clean[1])
    got = L.expert_product_forward(xs, w, offsets)
    dx, d = L.expert_product_backward(dys, xs, w, offsets)
    for x, y in ((got, ys), (dx, dxs), (d, dw)):
        plain.check_product(x, y)
    assert (got[:40] == 0).all() and (got[131:] == 0).all() and (dx[:40] == 0).all() and (dx[131:] == 0).all()
    assert (d[1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("stored", ["in_out", "out_in"])
@pytest.mark.parametrize("n,m,rows", [(128, 256, 5), (120, 200, 40), (264, 136, 400), (37, 50, 20)])
def test_nothing_reaches_another_expert(L, n, m, rows, stored, dtype):
    """NaN and infinities of one expert's rows and matrix stay with it, tails of rows and sums included."""
    xs, w, offsets, dys = inputs(3 * rows, n, m, [0, rows, 2 * rows, 3 * rows], dtype, stored)
    xs[:rows], dys[2 * rows:], w[0], w[2] = float("nan"), float("inf"), float("nan"), float("inf")
    mine = slice(rows, 2 * rows)
    one = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ys, dxs, dw = plain.products(xs[mine], w[1:2], one, dys[mine])
    got = L.expert_product_forward(xs, w, offsets)
    dx, d = L.expert_product_backward(dys, xs, w, offsets)
    plain.check_product(got[mine], ys)
    plain.check_product(dx[mine], dxs)
    plain.check_product(d[1:2], dw)
    assert not got[:rows].isfinite().any() and not dx[2 * rows:].isfinite().any() and d[0].isnan().all()


@pytest.mark.parametrize("n,m", [(64, 128), (72, 40)])
def test_strides_and_views(L, n, m):
    """Rows at a distance, matrices at a distance, starts that are no multiples of 16 bytes."""
    offsets = offsets_of([3, 0, 70, 20])
    rows = offsets[-1]
    xs, w, o, dys = inputs(rows, n, m, offsets, "bf16")
    want = check(L, xs, w, o, dys)
    wide_x = torch.full((rows, n + 24), float("nan"), device="cuda", dtype=xs.dtype)
    wide_y = torch.full((rows, m + 5), float("nan"), device="cuda", dtype=xs.dtype)
    wide_w = torch.full((8, n + 2, m + 16), float("nan"), device="cuda", dtype=xs.dtype)
    for ax, ay, aw in ((0, 0, 0), (8, 0, 8), (1, 3, 1)):
        x, y, matrices = wide_x[:, ax:ax + n], wide_y[:, ay:ay + m], wide_w[::2, :n, aw:aw + m]
        x.copy_(xs), y.copy_(dys), matrices.copy_(w)
        got = check(L, x, matrices, o, y)
        for a, b in zip(got, want):
            assert torch.allclose(a.float(), b.float(), atol=0.25, rtol=2 ** -6)
    # a matrix with neither side next to each other, rows that are columns, offsets at a distance
    x, y = xs.t().contiguous().t(), dys.t().contiguous().t()
    odd = torch.zeros(4, n, m, 2, device="cuda", dtype=xs.dtype)[..., 0]
    odd.copy_(w)
    spread = torch.zeros(len(offsets), 2, dtype=torch.int32, device="cuda")[:, 0]
    spread.copy_(o)
    check(L, x, odd, spread, y)
    # the same matrix for all experts
    shared = w[:1].expand(4, n, m)
    check(L, xs, shared, o, dys)


@pytest.mark.parametrize("stored", ["in_out", "out_in"])
def test_outputs_of_the_caller(L, stored):
    xs, w, offsets, dys = inputs(50, 64, 72, [0, 20, 50], "bf16", stored)
    want = check(L, xs, w, offsets, dys)
    ys, dx = torch.full_like(dys, 7), torch.full_like(xs, 7)
    wide = torch.full((2, 72, 80) if stored == "out_in" else (2, 64, 88), 7.0, device="cuda", dtype=w.dtype)
    dw = wide[:, :, :64].transpose(1, 2) if stored == "out_in" else wide[:, :, :72]
    version = ys._version, dw._version
    assert L.expert_product_forward(xs, w, offsets, out=ys) is ys
    got = L.expert_product_backward(dys, xs, w, offsets, out=(dx, dw))
    assert got[0] is dx and got[1] is dw and ys._version > version[0] and dw._version > version[1]
    for a, b in zip((ys, dx, dw), want):
        assert torch.equal(a, b)
    assert (wide[:, :, 64 if stored == "out_in" else 72:] == 7).all()  # what lies between its rows stays


def test_bad_offsets_stay_inside(L):
    """Offsets out of range are taken into it, and ranges that do not ascend are empty."""
    xs, w, _, dys = inputs(100, 64, 64, [0, 1, 2, 3, 4], "bf16")
    for offsets in ([-50, 30, 30, 400, 2 ** 31 - 1], [100, 100, 100, 100, 100], [-2 ** 31, -5, -1, 0, 0]):
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        check(L, xs, w, o, dys)
    falling = torch.tensor([80, 20, 60, 10, 5], dtype=torch.int32, device="cuda")
    L.expert_product_forward(xs, w, falling), L.expert_product_backward(dys, xs, w, falling)
    torch.cuda.synchronize()
    # ranges over one another, of many rows: more tiles than there could be
    xs, w, _, dys = inputs(5000, 264, 1032, list(range(21)), "bf16")
    over = torch.tensor([0, 5000] * 10 + [0], dtype=torch.int32, device="cuda")
    L.expert_product_forward(xs, w, over)
    _, dw = L.expert_product_backward(dys, xs, w, over)
    x, dy = xs.double(), dys.double()
    want = ((x.t() @ dy).cpu(), (x.t().abs() @ dy.abs()).cpu(), 5000)
    plain.check_product(dw[0], want), plain.check_product(dw[18], want)
    assert (dw[1::2] == 0).all()


def test_nothing_to_do(L):
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, w = torch.zeros(0, 16, device="cuda").bfloat16(), torch.ones(3, 16, 24, device="cuda").bfloat16()
    dy = torch.zeros(0, 24, device="cuda").bfloat16()
    assert L.expert_product_forward(x, w, o).shape == (0, 24)
    dx, dw = L.expert_product_backward(dy, x, w, o)
    assert dx.shape == (0, 16) and dw.shape == w.shape and (dw == 0).all()
    x, w = torch.zeros(5, 0, device="cuda").bfloat16(), torch.ones(3, 0, 24, device="cuda").bfloat16()
    assert (L.expert_product_forward(x, w, o) == 0).all() and L.expert_product_forward(x, w, o).shape == (5, 24)
    none, first = torch.ones(0, 16, 24, device="cuda").bfloat16(), o[:1]  # no expert at all: the rows are nobody's
    x, dy = torch.ones(5, 16, device="cuda").bfloat16(), torch.ones(5, 24, device="cuda").bfloat16()
    assert (L.expert_product_forward(x, none, first) == 0).all()
    dx, dw = L.expert_product_backward(dy, x, none, first)
    assert (dx == 0).all() and dw.shape == (0, 16, 24)


def test_refusals(L):
    xs, w, offsets, dys = inputs(20, 16, 24, [0, 10, 20], "bf16")
    for bad in (lambda: L.expert_product_forward(xs.float(), w, offsets), lambda: L.expert_product_forward(xs, w.float(), offsets),
                lambda: L.expert_product_forward(xs.double(), w.double(), offsets), lambda: L.expert_product_forward(xs.half(), w, offsets),
                lambda: L.expert_product_forward(dys, w, offsets), lambda: L.expert_product_forward(xs, w[0], offsets),
                lambda: L.expert_product_forward(xs, w, offsets[:2]), lambda: L.expert_product_forward(xs, w, offsets.long()),
                lambda: L.expert_product_forward(xs, w, offsets.cpu()), lambda: L.expert_product_forward(xs, w, offsets, out=xs),
                lambda: L.expert_product_backward(xs, xs, w, offsets), lambda: L.expert_product_backward(dys[:10], xs, w, offsets),
                lambda: L.expert_product_backward_weights(dys, xs, w, offsets, out=w[:1].expand(2, 16, 24)),
                lambda: L.expert_product(xs.cpu(), w, offsets)):
        with pytest.raises(L.LapsumError):
            bad()


def test_outputs_in_the_memory_of_inputs_are_refused(L):
    memory = torch.zeros(4000, device="cuda").bfloat16()
    xs, w, dys = memory[:320].view(20, 16), memory[320:832].view(2, 16, 16), memory[832:1152].view(20, 16)
    o = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    free = memory[1152:1472].view(20, 16)
    L.expert_product_forward(xs, w, o, out=free)
    for out in (xs, memory[8:328].view(20, 16), memory[824:1144].view(20, 16), memory[310:630].view(20, 16)):
        with pytest.raises(L.LapsumError):
            L.expert_product_forward(xs, w, o, out=out)
    for out in (memory[312:824].view(2, 16, 16), memory[1144:1656].view(2, 16, 16), memory[:512].view(2, 16, 16)):
        with pytest.raises(L.LapsumError):
            L.expert_product_backward_weights(dys, xs, w, o, out=out)
    L.expert_product_backward_weights(dys, xs, w, o, out=w)  # w itself is not read
    assert (memory == 0).all()


def test_differentiable(L):
    """Autograd: both gradients, one of them alone, shared rows, and a second derivative that is refused."""
    xs, w, offsets, dys = inputs(60, 64, 72, [0, 20, 20, 60], "fp16", "out_in")
    _, dxs, dw = plain.products(xs, w, offsets, dys)
    x, m = xs.clone().requires_grad_(), w.clone().requires_grad_()
    L.expert_product(x, m, offsets).backward(dys)
    plain.check_product(x.grad, dxs), plain.check_product(m.grad, dw)
    x.grad = None
    L.expert_product(x, w, offsets).backward(dys)
    plain.check_product(x.grad, dxs)
    m.grad = None
    L.expert_product(xs, m, offsets).backward(dys)
    plain.check_product(m.grad, dw)
    # an expanded upstream gradient
    x.grad = None
    L.expert_product(x, m, offsets).sum().backward()
    ones = plain.products(xs, w, offsets, torch.ones_like(dys))
    plain.check_product(x.grad, ones[1])
    y = L.expert_product(x, m, offsets)
    g, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    y = L.expert_product(x, m, offsets)
    offsets += 0  # written again before the backward
    with pytest.raises(RuntimeError):
        y.backward(dys)


def test_repeats_bit_for_bit_on_streams_and_in_a_graph(L):
    xs, w, offsets, dys = inputs(300, 256, 264, [0, 1, 150, 150, 300], "bf16")

    def run():
        return (L.expert_product_forward(xs, w, offsets), *L.expert_product_backward(dys, xs, w, offsets))
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        xs.mul_(-1), offsets.copy_(offsets.clone())  # other inputs, the same buffers
        want = run()


def test_both_fronts(L, monkeypatch):
    from sparse_selection_primitive_amd import hard
    for stored in ("in_out", "out_in"):
        xs, w, offsets, dys = inputs(50, 64, 72, [0, 20, 50], "bf16", stored)
        fast = (L.expert_product_forward(xs, w, offsets), *L.expert_product_backward(dys, xs, w, offsets))
        if hard._native is None:
            pytest.skip("the native front is not built")
        assert hard._native.expert_product_forward(xs, w, offsets) is not None
        assert hard._native.expert_product_forward(xs.double(), w, offsets) is None
        with monkeypatch.context() as m:
            m.setattr(hard, "_native", None)
            slow = (L.expert_product_forward(xs, w, offsets), *L.expert_product_backward(dys, xs, w, offsets))
        for a, b in zip(fast, slow):
            assert torch.equal(a, b) and a.stride() == b.stride()


def test_router_to_experts_and_back(L):
    """Route, plan, dispatch, two products and combine together, forward and gradients against the plain composition."""
    g = torch.Generator().manual_seed(3)
    tokens, experts, k, width, inner = 50, 8, 3, 64, 96
    x = torch.randn(tokens, width, generator=g).bfloat16().cuda().requires_grad_()
    logits = torch.randn(tokens, experts, generator=g).cuda().requires_grad_()
    up = (torch.randn(experts, width, inner, generator=g) / 8).bfloat16().cuda().requires_grad_()
    down = (torch.randn(experts, inner, width, generator=g) / 8).bfloat16().cuda().requires_grad_()
    dy = torch.randn(tokens, width, generator=g).bfloat16().cuda()
    weights, chosen = L.route(logits, k)
    offsets, slot, _ = L.dispatch_plan(chosen, experts)
    hidden = torch.relu(L.expert_product(L.dispatch(x, slot, offsets), up, offsets))
    y = L.combine(L.expert_product(hidden, down, offsets), weights, slot, offsets)
    y.backward(dy)
    # the same in 64 bits, the choice taken over
    leaves = [t.detach().double().cpu().requires_grad_() for t in (x, logits, up, down)]
    a, l, u, d = leaves
    p = torch.softmax(l, 1).gather(1, chosen.long().cpu())
    p = p / p.sum(1, keepdim=True)
    rows = []
    for t in range(tokens):
        rows.append(sum(p[t, j] * (torch.relu(a[t] @ u[e]) @ d[e]) for j, e in enumerate(chosen[t].tolist())))
    want = torch.stack(rows)
    want.backward(dy.double().cpu())
    # four roundings to bf16 on the way of values and gradients; sums of up to `width` terms of mixed sign
    for got, ref in ((y, want), (x.grad, a.grad), (logits.grad, l.grad), (up.grad, u.grad), (down.grad, d.grad)):
        err = (got.double().cpu() - ref).norm() / ref.norm()
        assert err < 4 * 2.0 ** -8, float(err)
