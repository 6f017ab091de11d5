"""How many of a weight's bits reach the output: outputs that cancel show them, since their own rounding is small.

Three entries a sequence, values chosen so that sum p v is far below sum p |v|.  Logits are below 2 and exact (one
product each), so a weight is off by the rounding of its logit in units of log2 (twice 2^-24 of at most 2.9), its power
(2^-23) and the quotient (2^-23): within 2^-21 of itself.  A product that held 16 bits of each weight would be off by
up to 2^-17 of them."""
import math

import pytest

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


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("width", [64, 96, 256])
@pytest.mark.parametrize("group", [1, 4, 16])
@pytest.mark.parametrize("capacity", [3, 5000])  # by one workgroup, and by splits
def test_weights_of_few_rows_keep_their_bits(L, capacity, group, width, dtype):
    batch = 64
    g = torch.Generator().manual_seed(group + width)
    z = (torch.randint(0, 256, (batch, 3), generator=g).double() / 128).to(TYPES[dtype]).double()
    p = torch.softmax(z, 1)
    # values of any size below the first; the second and third take up what is left
    v = torch.zeros(batch, 3, width, dtype=torch.float64)
    v[:, 0] = (1.0 + torch.rand(batch, width, generator=g).double()).to(TYPES[dtype]).double()
    for j in (1, 2):
        left = (p[:, :j, None] * v[:, :j]).sum(1)
        v[:, j] = (-left / p[:, j, None]).to(TYPES[dtype]).double()
    want, size = (p[..., None] * v).sum(1), (p[..., None] * v.abs()).sum(1)
    assert (want.abs() <= 2.0 ** -12 * size).double().mean() > 0.9
    k = torch.zeros(batch, 1, capacity, width, dtype=TYPES[dtype], device="cuda")
    vg = torch.zeros_like(k)
    k[:, 0, :3, 0] = z.to(TYPES[dtype]).cuda()
    vg[:, 0, :3] = v.to(TYPES[dtype]).cuda()
    q = torch.zeros(batch, 1, group, width, dtype=TYPES[dtype], device="cuda")
    q[..., 0] = 1.0
    n = torch.full((batch,), 3, dtype=torch.int32, device="cuda")
    out = L.cache_attend(q, k, vg, n, scale=1.0).double().cpu()
    err = (out[:, 0] - want[:, None]).abs()
    bound = 2.0 ** -21 * size + HALF_ULP[dtype] * want.abs() + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert (err <= bound[:, None]).all(), math.log2(float((err / size[:, None]).max()))
