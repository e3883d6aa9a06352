"""The serving operators where their inputs leave no rounding but the kernels' own, so that the bounds are those of a few
fp32 steps."""
import math
from decimal import Decimal, localcontext

import pytest
import torch

import serving_utils as su
from test_gpu_serving import BF16, F32, gen, normal, weights_call, within

pytestmark = pytest.mark.gpu
PI = Decimal("3.141592653589793238462643383279502884197169399375105820974944592307816")


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


def exact_turns(R, base, factor, orig_ctx, beta_fast=32.0, beta_slow=1.0):
    """Turns per position of every pair, to 60 digits."""
    with localcontext() as ctx:
        ctx.prec = 60
        out = []
        for k in range(R // 2):
            f = Decimal(base) ** (Decimal(-2 * k) / R) / (2 * PI)
            if orig_ctx:
                g = min(Decimal(1), max(Decimal(0), (orig_ctx * f - Decimal(beta_slow)) / (Decimal(beta_fast) - Decimal(beta_slow))))
                f = g * f + (1 - g) * f / Decimal(factor)
            else:
                f = f / Decimal(factor)
            out.append(f)
        return out


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("R,base,factor,orig", [(128, 10000.0, 1.0, 0), (64, 10000.0, 8.0, 0), (128, 500000.0, 16.0, 4096)])
def test_rope_angles_at_far_positions(v4a, half, R, base, factor, orig):
    """The reference's angle is exact, so the bound has no term that grows with the position but the frequencies' own: they
    are made by k products with base^(-2/R), each off by 3 x 2^-64 (2 of the power, 1 of the product), and up to a dozen
    more operations in 64-bit mantissas: (3 k + 12) 2^-64 relative.  At 2^40, with f_k <= base^(-2k/R) / 2 pi, that is at most
    16 x 2^-24 radians for these bases (12 at k = 0, 14 at most behind it).  An angle from a plain product in doubles is off by
    2^-13 there."""
    pos = [(1 << 40) - 1, -(1 << 40) + 12345, (1 << 39) + 7, (1 << 33) + 1, 1048575, 0]
    x = normal(gen(61), (1, len(pos), 2, R), F32)
    out = torch.empty_like(x, device="cuda")
    v4a.v4a_rope([(x.cuda(), out)], rope_dims=R, positions=torch.tensor([pos]).cuda(), half=half, rope_base=base, factor=factor, orig_ctx=orig)
    turns = exact_turns(R, base, factor, orig)
    with localcontext() as ctx:
        ctx.prec = 60
        ang = torch.tensor([[float((p * f) % 1) * 2 * math.pi for f in turns] for p in pos], dtype=torch.float64)[None, :, None]
    i0 = torch.arange(R // 2) if half else torch.arange(0, R, 2)
    i1 = i0 + (R // 2 if half else 1)
    a, b, ref = x[..., i0].double(), x[..., i1].double(), torch.empty(x.shape, dtype=torch.float64)
    ref[..., i0], ref[..., i1] = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
    made = torch.tensor([[2 * math.pi * abs(p) * float(f) * (3 * k + 12) * 2.0 ** -64 for k, f in enumerate(turns)] for p in pos], dtype=torch.float64)
    assert made.max() < 16 * su.U
    tol = su.rope_bound(x, ref, torch.zeros((1, len(pos))), R, 0)
    for i in (i0, i1):
        tol[..., i] += (a.abs() + b.abs()) * made[None, :, None]
    within(out, ref, tol, "far")
