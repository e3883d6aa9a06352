"""The serving operators where their inputs leave no rounding but the kernels' own, so that the bounds are those of a few
fp32 steps."""
import math

import pytest
import torch

import serving_utils as su
from test_gpu_serving import BF16, F32, gen, weights_call, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def v4a():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import compressed_sparse_long_v4a_b200 as v
    return v


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,H", [(64, 2), (256, 3)])
@pytest.mark.parametrize("size", [30, 900])
def test_weights_of_large_logits(v4a, dtype, d, H, size):
    """Whole numbers in q and own: every product and sum is exact in fp32, and so is the division by sqrt(d), 8 or 16.
    The lse are far from 0, as one or two keys of great weight make them.

    What is left of a term p = e^x, x = s - lse: one rounding of x, one of x log2 e and one of the constant (3 U |x|,
    relative to p), 2 ulp of the exponential (4 U); then the fp32 sum of n terms (n U of it)."""
    g = gen(60)
    rows = 70
    q = torch.randint(-3, 4, (2, 1, H, d), generator=g).float()
    own = torch.randint(-3, 4, (2, rows, d), generator=g).float()
    q[..., 0], own[..., 0] = 64.0, size * math.isqrt(d) / 64.0  # a whole number: moves every logit by `size`
    own[..., 0] = own[..., 0].round()
    s = torch.einsum("bthd,bnd->bthn", q.double(), own.double()) / math.sqrt(d)
    lse = (s.logsumexp(-1) + 0.1).float()
    assert float(lse.min()) > size / 2 and torch.equal(q, q.to(BF16).float()) and torch.equal(own, own.to(BF16).float())
    x = s - lse.double()[..., None]
    p = x.exp()
    ref = p.sum((1, 2))
    tol = (p * (3 * su.U * x.abs() + 4 * su.U + H * su.U)).sum((1, 2))
    c = dict(q=q.to(dtype), own=own.to(dtype), prefix=torch.zeros((0, d)), ctx_len=128 * rows, lens=[128 * rows] * 2, counts=[rows] * 2,
             entries=None)
    within(weights_call(v4a, c, lse, torch.zeros((2, rows)), 0.0), ref, tol, "weights")
