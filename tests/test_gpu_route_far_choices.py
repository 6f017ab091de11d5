"""Routing where the choice lies far below the row's maximum: a bias, or limited groups, can leave out the experts of
the largest logits.  The weights of a renormalised softmax are the softmax of the chosen logits, however far they lie
below the others; forward and gradient are those of one function.  Tolerances as in test_gpu_route."""
import math

import pytest

import hard_plain as plain
import test_gpu_route as r

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_selection_primitive_amd as lib
    lib.load_library()
    return lib


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("experts,k", [(12, 4), (64, 6), (256, 8), (300, 20), (1024, 3)])
@pytest.mark.parametrize("below", [80, 88, 104, 150, 400])
def test_choice_by_the_bias(L, below, experts, k, dtype):
    """Experts `below` under the maximum: their shares of the whole softmax fall under fp32's range from about 87 on."""
    x = torch.full((4, experts), -float(below), dtype=torch.float64)
    bias = torch.full((experts,), 2.0, dtype=torch.float64)
    x[:, 1] = 0.0  # the maximum, which the bias rules out
    bias[1] = 0.0
    # the choice goes by the bias alone (shares this small round away in the sum): distinct values, so that no tie is near
    bias[2:2 + k] += torch.arange(k, 0, -1).double() / 8
    step = 0.5 if below < 128 else (1.0 if below < 256 else 2.0)  # bf16 numbers
    x[1, 2:2 + k] -= step * torch.arange(k)
    x[2, 2] += 4 * step
    x[3, 2:2 + k:2] -= 40.0  # some fall behind the others
    assert torch.equal(x, x.to(r.TYPES[dtype]).double())
    r.check(L, x, k, bias, dtype, scale=2.5)
    xt = x.to(r.TYPES[dtype]).cuda()
    w, c = L.route_forward(xt, k, bias.float().cuda())
    assert c.cpu().tolist() == [list(range(2, 2 + k))] * 4
    want = torch.softmax(x[:, 2:2 + k], 1)
    spread = float((x[:, 2:2 + k].amax(1) - x[:, 2:2 + k].amin(1)).max())
    assert ((w.double().cpu() - want).abs() <= (16 + 4 * spread) * 2.0 ** -24 * want + 1e-37).all()
    assert ((w.double().cpu().sum(1) - 1.0).abs() <= (k + 8) * 2.0 ** -24).all()


@pytest.mark.parametrize("experts,groups", [(32, 4), (60, 4), (256, 8)])
def test_choice_by_the_groups(L, experts, groups):
    """The maximum stands alone in its group, which counts as one without experts: the others are far below it."""
    size = experts // groups
    x = torch.full((2, experts), -200.0, dtype=torch.float64)
    x[:, 1:size] = -math.inf
    x[:, 0] = 0.0
    x[1, size + 2] = -198.0
    w, c = L.route_forward(x.float().cuda(), 3, groups=groups, top_groups=1)
    # every share is 0 in fp32, so the choice is the first open group's first three
    assert c.cpu().tolist() == [[size, size + 1, size + 2]] * 2
    want = torch.softmax(x[:, size:size + 3], 1)
    assert ((w.double().cpu() - want).abs() <= 24 * 2.0 ** -24 * want).all()


def test_gradient_is_the_forwards(L):
    """Differences of the kernel's own weights, by a step that fp32 resolves."""
    x = torch.full((1, 16), -150.0)
    x[0, 0] = 0.0
    x[0, 5], x[0, 9] = -149.0, -151.5
    bias = torch.zeros(16)
    bias[[3, 5, 9]] = torch.tensor([4.0, 3.0, 2.0])
    dw = torch.tensor([[1.0, -2.0, 0.5]], device="cuda")

    def weights(z):
        w, c = L.route_forward(z.cuda(), 3, bias.cuda())
        assert c.tolist() == [[3, 5, 9]]
        return (w.double() * dw).sum()
    _, c = L.route_forward(x.cuda(), 3, bias.cuda())
    dx = L.route_backward(dw, x.cuda(), c)
    h = 2.0 ** -6  # exact in fp32 at this size; the difference is off by h^2 and by 2^-23 / h of weights below 4
    for i in range(16):
        e = torch.zeros_like(x)
        e[0, i] = h
        assert float((weights(x + e) - weights(x - e)) / (2 * h)) == pytest.approx(float(dx[0, i]), abs=4 * h * h + 1e-4)


@pytest.mark.parametrize("experts,groups", [(8, 2), (64, 8), (60, 4), (256, 8)])
def test_group_score_past_the_range_is_a_score(L, experts, groups):
    """Two experts whose c are each below half of the lowest fp32 number are available: their group, whose sum is past
    the range, comes before one without experts."""
    size = experts // groups
    x, bias = r.grid_logits(5, experts, 7), torch.zeros(experts)
    x[:, :-size] = -math.inf
    bias[-size:] = -3.0e38
    _, c = L.route_forward(x.float().cuda(), 2, bias.cuda(), score="sigmoid", groups=groups, top_groups=1)
    assert c.cpu().tolist() == [[experts - size, experts - size + 1]] * 5  # c are equal in fp32


@pytest.mark.parametrize("experts,groups", [(8, 2), (64, 8), (60, 4), (256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_mask_of_the_lowest_number_is_one_of_minus_infinity(L, score, experts, groups):
    """In a bias, the lowest fp32 number takes an expert out as -inf does, for its group's score as well."""
    size = experts // groups
    x = r.grid_logits(6, experts, 13).float().cuda()
    for left in ([], [1], [1, 2], [0, 3]):  # the experts that stay in the last group; the other groups have none
        out = []
        for mask in (-math.inf, torch.finfo(torch.float32).min):
            bias = torch.full((experts,), mask)
            bias[[experts - size + i for i in left]] = 0.25
            out.append(L.route_forward(x, 2, bias.cuda(), score=score, groups=groups, top_groups=1))
        assert torch.equal(out[0][1], out[1][1]) and torch.equal(out[0][0], out[1][0])
        want = [experts - size + i for i in left] if len(left) > 1 else [-1, -1]
        assert sorted(out[0][1][0].tolist()) == want


@pytest.mark.parametrize("experts", [64, 65, 130, 200, 260])
def test_places_past_the_last_group(L, experts):
    """Groups of one expert, as many as there can be: a wave's last places name groups that do not exist."""
    groups = max(g for g in range(1, 65) if experts % g == 0)
    x, bias = r.grid_logits(9, experts, experts), r.grid_bias(experts, 2)
    kw = dict(score="sigmoid", groups=groups, top_groups=max(1, groups - 1))
    keep = r.settled(x, bias, kw)
    r.check(L, x[keep], min(8, experts // groups * kw["top_groups"]), bias, **kw)
