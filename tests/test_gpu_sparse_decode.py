"""The decode loop of examples/sparse_decode.py: the hard selections together.

With a budget that is never reached the loop's attention is that of the whole
history, whose plain form is computed here; with a small one the cache holds
its budget, the protected entries, and accounts that add up: every step adds
one unit of weight per query head.  Tolerances: inputs are bf16, so an
output of attention is within 2^-8 of the values' mean size, and the block's
output, a sum of a few such terms through two products, within 2^-5 of its size."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_decode
    return sparse_decode


def plain_attention(block, history, x):
    """Attention of the newest token over the whole history [batch, tokens, width], float64."""
    s = block.s
    k, v = (t.double() for t in block.keys_values(history))
    q = block.queries(x[:, None])[:, 0].double()
    g = s.heads // s.kv_heads
    z = torch.matmul(k.repeat_interleave(g, 1), q[..., None])[..., 0] * s.head_width ** -0.5
    return torch.matmul(torch.softmax(z, 2)[:, :, None], v.repeat_interleave(g, 1))[:, :, 0]


def test_without_eviction_it_is_attention_over_everything(E):
    s = E.Shape(batch=2, prompt=50, budget=90, window=8)
    block = E.Block(s)
    g = torch.Generator(device="cuda").manual_seed(3)
    history = torch.randn(2, 50, s.width, generator=g, device="cuda").bfloat16()
    with torch.no_grad():
        cache = E.prefill(block, history)
        for _ in range(5):
            x = torch.randn(2, s.width, generator=g, device="cuda").bfloat16()
            history = torch.cat([history, x[:, None]], 1)
            cache.append(*block.keys_values(x[:, None]))
            out = cache.attend(block.queries(x[:, None]))[:, 0].double()
            want = plain_attention(block, history, x)
            assert (out - want).abs().max() <= 2.0 ** -8 * (1.0 + want.abs().max())
            cache.evict(s.budget)
    assert cache.lengths.tolist() == [55, 55]
    # each of the 8 window tokens and 5 steps gave one unit of weight per query head
    total = cache.account[:, :, :55].double().sum((1, 2))
    assert (total - 13 * s.heads).abs().max() <= 1e-3


def test_with_a_budget(E):
    s = E.Shape(batch=3, prompt=200, budget=64, window=8, sinks=2, recent=16)
    block = E.Block(s, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    with torch.no_grad():
        cache = E.prefill(block, torch.randn(3, 200, s.width, generator=g, device="cuda").bfloat16())
        for i in range(30):
            y = E.step(block, cache, torch.randn(3, s.width, generator=g, device="cuda").bfloat16())
            assert torch.isfinite(y).all()
    assert cache.lengths.tolist() == [64] * 3 and cache.next_position.tolist() == [230] * 3
    for b in range(3):
        for h in range(s.kv_heads):
            held = set(cache.positions[b, h, :64].tolist())
            assert len(held) == 64 and held >= {0, 1} | set(range(214, 230))


def test_training_step(E):
    """Gradients through route, dispatch and combine against differences of the loss along a direction."""
    s = E.Shape(width=64, experts=8, k=2)
    block = E.Block(s, 7)
    block.router = block.router.float().requires_grad_(True)
    block.up, block.down = block.up.float(), block.down.float()
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(40, 64, generator=g, device="cuda")
    up = torch.randn(40, 64, generator=g, device="cuda")
    bias = block.bias.clone()

    def loss():
        block.bias = bias.clone()
        return (block.mixture(x) * up).double().sum()

    loss().backward()
    grad = block.router.grad.double()
    d = torch.randn(block.router.shape, generator=g, device="cuda")
    d /= d.norm()
    with torch.no_grad():
        base, h = block.router.clone(), 1e-3
        block.router = base + h * d
        up_loss = loss()
        block.router = base - h * d
        down_loss = loss()
    slope = float((up_loss - down_loss) / (2 * h))
    # fp32 losses of size ~1e2 give the difference to 1e-5 / h, and the step's curvature to h^2
    assert slope == pytest.approx(float((grad * d).sum()), abs=2e-2 * float(grad.norm()) + 2e-2)


def test_main(E, capsys):
    cache, x = E.main(["--steps", "8"])
    assert torch.isfinite(x).all() and "8 steps" in capsys.readouterr().out
