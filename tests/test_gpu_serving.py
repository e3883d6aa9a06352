"""Rotary positions, attention over a shared prefix, accumulated attention weights and eviction on the GPU, against
plain 64-bit forms; the bounds are derived in serving_utils.py."""
import math

import pytest
import torch

import serving_utils as su

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def v4a():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import compressed_sparse_long_v4a_b200 as v
    return v


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, dtype):
    return torch.randn(shape, generator=g).to(dtype)


def within(got, ref, tol, what=""):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    assert torch.equal(got.isinf(), ref.isinf()), what
    ok = torch.isfinite(ref)
    bad = ((got - ref).abs() > tol) & ok
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: {got[i]} for {ref[i]}, bound {tol[i]}")


# ------------------------------------------------------------------ rotary positions

ROPE = [
    # dtype, B, T, H, d, R, offset (None: last), half
    (BF16, 2, 3, 64, 512, 64, None, False), (BF16, 1, 5, 4, 128, 128, None, True), (F32, 2, 7, 3, 128, 64, 0, True),
    (F32, 1, 1, 1, 64, 64, None, False), (BF16, 2, 2, 5, 96, 48, 40, True), (F32, 3, 2, 2, 70, 22, 13, False),
    (BF16, 1, 3, 7, 66, 66, None, True), (F32, 1, 2, 1, 512, 512, None, False), (BF16, 1, 700, 2, 64, 16, 8, False),
    (BF16, 2, 2, 2, 64, 2, 1, True)]


@pytest.mark.parametrize("dtype,B,T,H,d,R,off,half", ROPE)
@pytest.mark.parametrize("inverse,in_place", [(False, False), (True, True)])
def test_rope(v4a, dtype, B, T, H, d, R, off, half, inverse, in_place):
    g = gen(7)
    x = normal(g, (B, T, H, d), dtype)
    pos = torch.randint(0, 1 << 20, (B, T), generator=g)
    o = d - R if off is None else off
    ref = su.rope_ref(x, pos, R, o, half, inverse)
    dx = x.cuda()
    out = dx if in_place else torch.full_like(dx, 7.0)
    v4a.v4a_rope([(dx, out)], rope_dims=R, positions=pos.cuda(), rope_offset=off, half=half, inverse=inverse)
    within(out, ref, su.rope_bound(x, ref, pos, R, o, rounding=su.BF if dtype == BF16 else su.U), "rope")
    keep = [i for i in range(d) if not o <= i < o + R]
    assert torch.equal(out.cpu()[..., keep], x[..., keep])  # copied, to the bit


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("factor,orig,scale", [(8.0, 0, 1.0), (16.0, 4096, 0.1 * math.log(16.0) + 1.0), (0.5, 0, 2.0)])
def test_rope_scaled_and_far(v4a, half, factor, orig, scale):
    g = gen(8)
    x = normal(g, (1, 6, 2, 128), F32)
    pos = torch.tensor([[0, 1, 65537, (1 << 31) + 12345, (1 << 40) - 1, -17]])
    ref = su.rope_ref(x, pos, 128, 0, half, False, scale, factor=factor, orig_ctx=orig)
    out = torch.empty_like(x, device="cuda")
    v4a.v4a_rope([(x.cuda(), out)], rope_dims=128, positions=pos.cuda(), half=half, factor=factor, orig_ctx=orig, out_scale=scale)
    within(out, ref, su.rope_bound(x, ref, pos, 128, 0, scale), "scaled")


def test_rope_streams_strides_and_steps(v4a):
    # a decode step: heads cut out of a fused projection, the K=V row, indexer heads stored [B][H][T][d]; compressed
    # entries' positions come as a start and a step
    g = gen(9)
    B, T = 3, 4
    fused = normal(g, (B, T, 9, 128), BF16)
    kv = normal(g, (B, T, 128), BF16)
    idx = normal(g, (B, 5, T, 64), BF16)
    pos = (1000 + 128 * torch.arange(T)).expand(B, T)
    df, dk, di = fused.cuda(), kv.cuda(), idx.cuda()
    out = [torch.zeros((B, T, 4, 128), dtype=BF16, device="cuda"), torch.zeros((B, T + 2, 128), dtype=BF16, device="cuda"),
           torch.zeros((B, 5, T, 64), dtype=BF16, device="cuda")]
    v4a.v4a_rope([(df[:, :, 2:6], out[0]), (dk, out[1][:, 1:T + 1]), (di.transpose(1, 2), out[2].transpose(1, 2))], rope_dims=64,
                 pos0=1000, pos_step=128)
    for x, y in ((fused[:, :, 2:6], out[0]), (kv[:, :, None], out[1][:, 1:T + 1, None]), (idx.transpose(1, 2), out[2].transpose(1, 2))):
        off = x.shape[-1] - 64
        ref = su.rope_ref(x, pos, 64, off)
        within(y, ref, su.rope_bound(x, ref, pos, 64, off, rounding=su.BF), "stream")
    assert (out[1][:, 0] == 0).all() and (out[1][:, T + 1] == 0).all()


def test_rope_gradient(v4a):
    # the gradient of sum(out * w): the formula's by automatic differentiation in 64 bits, and differences
    g = gen(10)
    x, w = normal(g, (1, 3, 2, 64), F32), normal(g, (1, 3, 2, 64), F32)
    pos = torch.tensor([[5, 700, 65000]])
    kw = dict(factor=4.0, orig_ctx=2048, out_scale=1.25)
    dw = torch.empty_like(w, device="cuda")
    v4a.v4a_rope([(w.cuda(), dw)], rope_dims=48, positions=pos.cuda(), inverse=True, **{**kw, "half": True})

    def value(z):
        f = torch.tensor(su.rope_frequencies(48, factor=4.0, orig_ctx=2048), dtype=torch.float64)
        ang = (pos.double()[..., None] * f)[:, :, None]
        a, b = z[..., 16:40], z[..., 40:]
        y = torch.cat((z[..., :16], 1.25 * (a * ang.cos() - b * ang.sin()), 1.25 * (b * ang.cos() + a * ang.sin())), -1)
        return (y * w.double()).sum()

    z = x.double().requires_grad_()
    value(z).backward()
    bound = su.rope_bound(w, z.grad, pos, 48, 16, 1.25)
    within(dw, z.grad, bound, "gradient")
    for at in ((0, 0, 0, 3), (0, 1, 1, 20), (0, 2, 0, 63)):  # linear in x: a difference is exact to 64-bit rounding
        h = torch.zeros_like(z.detach())
        h[at] = 1.0
        diff = (value(z.detach() + h) - value(z.detach() - h)) / 2
        assert abs(diff - dw.cpu().double()[at]) <= bound[at] + 1e-9


def test_rope_then_attention_reads_the_rotated_query(v4a):
    # the attention kernels request their first query early: it must be the rotated one, call after call
    g = gen(11)
    B, H, d, N = 4, 64, 512, 700
    ent = normal(g, (B, N, d), BF16).cuda()
    ring = torch.zeros((B, 1, d), dtype=BF16, device="cuda")
    qs = [normal(g, (B, 1, H, d), BF16).cuda() for _ in range(6)]
    want = []
    for i, q in enumerate(qs):
        r = torch.empty_like(q)
        v4a.v4a_rope([(q, r)], rope_dims=64, pos0=1000 * i)
        torch.cuda.synchronize()
        o = torch.empty((B, 1, H, d), device="cuda")
        v4a.v4a_hca_attend(r, ent, ring, N * 128 - 1, o, m=128, window=0, ctx_len=N * 128)
        want.append(o)
    r = torch.empty_like(qs[0])
    got = [torch.empty_like(want[0]) for _ in qs]
    for _ in range(20):
        for i, q in enumerate(qs):
            v4a.v4a_rope([(q, r)], rope_dims=64, pos0=1000 * i)
            v4a.v4a_hca_attend(r, ent, ring, N * 128 - 1, got[i], m=128, window=0, ctx_len=N * 128)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ shared-prefix attention

def shared_case(dtype, B, T, H, d, Np, rows, W, m=128, ragged=True, evicted=False, dead=(), seed=1, ring_rows=None):
    g = gen(seed)
    c = dict(m=m, W=W)
    c["q"], c["prefix"], c["own"] = normal(g, (B, T, H, d), dtype), normal(g, (Np, d), dtype), normal(g, (B, rows, d), dtype)
    c["ring"] = normal(g, (B, ring_rows or max(1, W + T - 1), d), dtype)
    counts = [int(torch.randint(0, rows + 1, (1,), generator=g)) if ragged and b else rows for b in range(B)]
    entries, lens = None, []
    if evicted:
        entries = [sorted((torch.randperm(2 * rows, generator=g)[:rows] + Np).tolist()) for _ in range(B)]
    for b in range(B):
        top = Np + (2 * rows if evicted else counts[b])
        # not every own entry need be seen: with few tokens behind the last chunk, early queries miss the newest entry
        lens.append(max(m * Np + T, m * top + int(torch.randint(0, m, (1,), generator=g))))
        if b in dead:
            lens[b], counts[b] = 0, 0
    c.update(counts=counts, entries=entries, lens=lens, ctx_len=max(m * (Np + 2 * rows + 1) + T, 1))
    return c


def attend(v4a, c, out_dtype=None, sink=None, rope_dims=0, status=None, lse=True, **kw):
    q = c["q"].cuda()
    out = torch.full(q.shape, 7.0, dtype=out_dtype or q.dtype, device="cuda")
    l = torch.full(q.shape[:3], 7.0, device="cuda") if lse else None
    v4a.v4a_hca_attend_shared(
        q, c["prefix"].cuda() if c["prefix"].shape[0] else None, c["own"].cuda() if c["own"].shape[1] else None,
        c["ring"].cuda() if c["W"] else None, out, m=c["m"], window=c["W"], ctx_len=c["ctx_len"],
        ctx_lens=torch.tensor(c["lens"]).cuda(), own_count=torch.tensor(c["counts"], dtype=torch.int32).cuda(),
        own_entry=torch.tensor(c["entries"], dtype=torch.int32).cuda() if c["entries"] is not None else None, lse=l,
        sink=sink.cuda() if sink is not None else None, rope_dims=rope_dims, dev_status=status, **kw)
    return out, l


def check_shared(v4a, c, out_dtype=None, sink=None, rope_dims=0):
    bf = c["q"].dtype == BF16
    odt = out_dtype or c["q"].dtype
    ref, lse, tol, tol_l = su.shared_ref(c["q"], c["prefix"], c["own"], c["ring"], lens=c["lens"], counts=c["counts"],
                                         entries=c["entries"], m=c["m"], W=c["W"], sink=sink, rope_dims=rope_dims,
                                         p_rounding=su.BF if bf else su.U, out_rounding=su.BF if odt == BF16 else su.U)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    out, l = attend(v4a, c, out_dtype, sink, rope_dims, status)
    assert int(status) == 0
    within(out, ref, tol, "out")
    within(l, lse, tol_l, "lse")
    return out, l


SHARED = [
    # dtype, B, T, H, d, Np, rows, W
    (F32, 3, 1, 16, 128, 100, 5, 128), (F32, 1, 1, 1, 64, 1, 1, 1), (F32, 2, 3, 5, 64, 33, 40, 7), (F32, 2, 2, 17, 256, 65, 3, 0),
    (F32, 1, 2, 4, 512, 31, 70, 64), (BF16, 3, 2, 8, 64, 200, 17, 128), (BF16, 2, 1, 3, 512, 40, 9, 16), (BF16, 2, 1, 40, 128, 0, 50, 33),
    (BF16, 4, 1, 64, 512, 300, 70, 128), (BF16, 1, 1, 64, 512, 1, 1, 1), (BF16, 5, 2, 8, 512, 129, 66, 100), (BF16, 2, 3, 128, 512, 64, 3, 0),
    (BF16, 3, 1, 16, 512, 500, 0, 64), (BF16, 2, 1, 32, 512, 0, 130, 128), (BF16, 1, 4, 4, 512, 700, 10, 130), (BF16, 2, 1, 64, 512, 0, 0, 5),
    (BF16, 9, 1, 12, 512, 63, 64, 65), (BF16, 2, 1, 192, 512, 192, 5, 128)]


@pytest.mark.parametrize("dtype,B,T,H,d,Np,rows,W", SHARED)
@pytest.mark.parametrize("evicted", [False, True])
def test_shared_attention(v4a, dtype, B, T, H, d, Np, rows, W, evicted):
    check_shared(v4a, shared_case(dtype, B, T, H, d, Np, rows, W, evicted=evicted, ring_rows=256 if W else None))


@pytest.mark.parametrize("dtype,H,d", [(F32, 4, 128), (BF16, 64, 512), (BF16, 8, 512)])
def test_shared_attention_sink_rotation_fp32_output(v4a, dtype, H, d):
    c = shared_case(dtype, 3, 2, H, d, 90, 20, 64, seed=3)
    sink = torch.randn((H,), generator=gen(4)) * 3
    check_shared(v4a, c, sink=sink, rope_dims=64)
    check_shared(v4a, c, out_dtype=F32, rope_dims=d)


@pytest.mark.parametrize("dtype,H,d", [(F32, 6, 64), (BF16, 64, 512), (BF16, 16, 512)])
def test_shared_attention_padded_batch_and_empty_rows(v4a, dtype, H, d):
    c = shared_case(dtype, 4, 2, H, d, 40, 12, 32, dead=(0, 2), seed=5)
    out, lse = check_shared(v4a, c, sink=torch.ones(H))
    assert (out[0] == 0).all() and (out[2] == 0).all() and torch.isneginf(lse[0]).all()
    # a sequence shorter than n_q: its first query lies before position 0 (no prefix, so nothing is at fault)
    c = shared_case(dtype, 2, 3, H, d, 0, 2, 4, seed=6)
    c["lens"], c["counts"] = [2, 1], [0, 0]
    out, lse = check_shared(v4a, c)
    assert (out[0, 0] == 0).all() and (out[1, :2] == 0).all() and torch.isfinite(lse[0, 1:]).all()
    # no candidates at all: a sink alone leaves zeros
    c = shared_case(dtype, 2, 1, H, d, 0, 3, 0, seed=6)
    c["counts"] = [0, 0]
    out, lse = attend(v4a, c, sink=torch.ones(H))
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,H,d", [(F32, 4, 128), (BF16, 64, 512), (BF16, 8, 512)])
def test_shared_attention_masked_places_may_hold_anything(v4a, dtype, H, d, bad):
    c = shared_case(dtype, 3, 2, H, d, 70, 70, 48, dead=(1,), seed=7, evicted=True, ring_rows=64)
    c["entries"][0][3] = -1  # an empty slot
    clean, lse = check_shared(v4a, c)
    d2 = dict(c)
    d2["own"], d2["ring"], d2["q"] = c["own"].clone(), c["ring"].clone(), c["q"].clone()
    for b in range(3):
        d2["own"][b, c["counts"][b]:] = bad
        used = {p % 64 for p in range(max(0, c["lens"][b] - 2 - 48 + 1), c["lens"][b])}
        d2["ring"][b, [r for r in range(64) if r not in used]] = bad
        last = c["lens"][b] - 1
        for i in range(c["counts"][b]):
            if not 0 <= 128 * (c["entries"][b][i] + 1) <= last + 1 or c["entries"][b][i] < 0:
                d2["own"][b, i] = bad
    d2["q"][1] = bad  # the padded sequence
    out, lse2 = attend(v4a, d2)
    assert torch.equal(out, clean) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,H,d", [(F32, 4, 128), (BF16, 64, 512)])
def test_shared_attention_nan_stays_in_its_sequence(v4a, dtype, H, d):
    c = shared_case(dtype, 3, 1, H, d, 50, 9, 16, ragged=False, seed=8)
    clean, _ = attend(v4a, c)
    for key, at in (("own", (1, 4)), ("ring", (1,)), ("q", (1,))):
        d2 = {**c, key: c[key].clone()}
        d2[key][at] = math.nan
        out, lse = attend(v4a, d2)
        assert torch.equal(out[[0, 2]], clean[[0, 2]]), key
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all(), key


@pytest.mark.parametrize("dtype,H,d", [(F32, 4, 128), (BF16, 64, 512), (BF16, 8, 512)])
def test_shared_attention_reports_bad_lengths_and_counts(v4a, dtype, H, d):
    for what, i, value in (("lens", 1, -3), ("lens", 1, 1 << 40), ("counts", 1, -1), ("counts", 1, 10), ("lens", 1, 128 * 20 - 1)):
        c = shared_case(dtype, 3, 1, H, d, 20, 9, 16, seed=9)
        good, _ = attend(v4a, c)
        c[what][i] = value
        status = torch.zeros((1,), dtype=torch.int32, device="cuda")
        out, lse = attend(v4a, c, status=status)
        assert int(status) == 4, (what, value)
        assert torch.equal(out[[0, 2]], good[[0, 2]])
        if what == "lens":
            assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
        else:
            c["counts"][1] = min(max(value, 0), 9)
            clamped, _ = attend(v4a, c)
            assert torch.equal(out[1], clamped[1])


def test_shared_attention_agrees_with_the_contiguous_call(v4a):
    # one sequence's prefix and own entries side by side are v4a_hca_attend's entries
    c = shared_case(BF16, 1, 1, 64, 512, 200, 56, 128, ragged=False, seed=10)
    L = c["lens"][0] = c["ctx_len"] = 128 * 256 + 5
    ref, _, tol, _ = su.shared_ref(c["q"], c["prefix"], c["own"], c["ring"], lens=[L], counts=[56], entries=None, m=128, W=128,
                                   p_rounding=su.BF)
    tok = c["ring"][:, [p % c["ring"].shape[1] for p in range(L - 128, L)]].contiguous().cuda()
    plain = torch.empty((1, 1, 64, 512), device="cuda")
    v4a.v4a_hca_attend(c["q"].cuda(), torch.cat((c["prefix"], c["own"][0]))[None].contiguous().cuda(), tok, L - 128, plain, m=128,
                       window=128, ctx_len=L)
    out, _ = attend(v4a, c, out_dtype=F32)
    within(out, ref, tol)
    within(plain, ref, 2 * tol)  # this call also sums rounded probabilities


@pytest.mark.parametrize("dtype,B,T,H,d", [(F32, 2, 1, 16, 128), (BF16, 6, 1, 64, 512), (BF16, 20, 1, 8, 512)])
def test_shared_attention_repeats_to_the_bit_on_any_stream_and_captured(v4a, dtype, B, T, H, d):
    c = shared_case(dtype, B, T, H, d, 900, 30, 128, seed=11)
    first, lse = attend(v4a, c)
    dev = {k: c[k].cuda() for k in ("q", "prefix", "own", "ring")}
    lens, cnt = torch.tensor(c["lens"]).cuda(), torch.tensor(c["counts"], dtype=torch.int32).cuda()
    ws = torch.full((v4a.v4a_shared_workspace_size(batch=B, n_q=T, heads=H, d=d, n_prefix=900, own_rows=30, window=128, dtype=dtype),),
                    255, dtype=torch.uint8, device="cuda")  # NaN in every partial: nothing is read before it is written
    out, l = torch.empty_like(dev["q"]), torch.empty_like(lse)

    def call(**kw):
        v4a.v4a_hca_attend_shared(dev["q"], dev["prefix"], dev["own"], dev["ring"], out, m=128, window=128, ctx_len=c["ctx_len"],
                                  ctx_lens=lens, own_count=cnt, lse=l, workspace=ws, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(out, first) and torch.equal(l, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(2):
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(l, lse)
    dev["q"].copy_(-dev["q"])  # other inputs in the same buffers
    graph.replay()
    torch.cuda.synchronize()
    c["q"] = -c["q"]
    assert torch.equal(out, attend(v4a, c)[0])


# ------------------------------------------------------------------ weights

WEIGHTS = [
    # dtype, B, T, H, d, Np, rows
    (F32, 3, 2, 16, 128, 6, 50), (F32, 1, 1, 1, 64, 0, 1), (F32, 2, 1, 20, 256, 3, 33), (BF16, 2, 1, 5, 64, 2, 40),
    (BF16, 2, 1, 64, 512, 0, 300), (BF16, 3, 2, 8, 512, 7, 129), (BF16, 1, 3, 128, 512, 1, 64), (BF16, 2, 5, 16, 512, 0, 1),
    (BF16, 1, 1, 12, 512, 2, 257)]


def weights_call(v4a, c, lse, w, decay, **kw):
    out = torch.full_like(w, 7.0, device="cuda")
    v4a.v4a_attend_weights(c["q"].cuda(), c["own"].cuda(), lse.cuda(), w.cuda(), out, m=128, ctx_len=c["ctx_len"],
                           n_prefix=c["prefix"].shape[0], ctx_lens=torch.tensor(c["lens"]).cuda(),
                           own_count=torch.tensor(c["counts"], dtype=torch.int32).cuda(),
                           own_entry=torch.tensor(c["entries"], dtype=torch.int32).cuda() if c["entries"] is not None else None,
                           decay=decay, **kw)
    return out


@pytest.mark.parametrize("dtype,B,T,H,d,Np,rows", WEIGHTS)
@pytest.mark.parametrize("evicted,decay", [(False, 1.0), (True, 0.75), (True, 0.0)])
def test_attend_weights(v4a, dtype, B, T, H, d, Np, rows, evicted, decay):
    c = shared_case(dtype, B, T, H, d, Np, rows, 0, evicted=evicted, seed=12)
    g = gen(13)
    w = torch.rand((B, rows), generator=g) * 5
    lse = torch.randn((B, T, H), generator=g) + 3
    lse[0, 0, 0] = -math.inf
    ref, tol = su.weights_ref(c["q"], c["own"], lse, w, n_prefix=Np, lens=c["lens"], counts=c["counts"], entries=c["entries"], m=128,
                              decay=decay)
    out = weights_call(v4a, c, lse, w, decay)
    held = ~torch.isnan(ref)
    assert (out.cpu()[~held] == 7.0).all()  # beyond the count: left as it was
    within(torch.where(held.cuda(), out, 0.0), torch.where(held, ref, 0.0), tol, "weights")
    assert torch.equal(out, weights_call(v4a, c, lse, w, decay))  # in a fixed order


@pytest.mark.parametrize("dtype,H,d", [(F32, 4, 128), (BF16, 64, 512)])
def test_attend_weights_masked_places_in_place_and_captured(v4a, dtype, H, d):
    c = shared_case(dtype, 3, 2, H, d, 4, 140, 0, evicted=True, dead=(1,), seed=14)
    g = gen(15)
    w, lse = torch.rand((3, 140), generator=g), torch.randn((3, 2, H), generator=g)
    clean = weights_call(v4a, c, lse, w, 1.0)
    d2 = {**c, "own": c["own"].clone(), "q": c["q"].clone()}
    d2["q"][1] = math.nan
    for b in range(3):
        d2["own"][b, c["counts"][b]:] = math.nan
    assert torch.equal(weights_call(v4a, d2, lse, w, 1.0), clean)
    # in place, and as a captured pair of steps
    q, own, acc, l = c["q"].cuda(), c["own"].cuda(), w.cuda(), lse.cuda()
    kw = dict(m=128, ctx_len=c["ctx_len"], n_prefix=4, ctx_lens=torch.tensor(c["lens"]).cuda(),
              own_count=torch.tensor(c["counts"], dtype=torch.int32).cuda(), own_entry=torch.tensor(c["entries"], dtype=torch.int32).cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v4a.v4a_attend_weights(q, own, l, acc, acc, **kw)
        v4a.v4a_attend_weights(q, own, l, acc, acc, **kw)
    graph.replay()
    torch.cuda.synchronize()
    twice = weights_call(v4a, c, lse, torch.where(torch.arange(140) < torch.tensor(c["counts"])[:, None], clean.cpu(), w), 1.0)
    held = (torch.arange(140) < torch.tensor(c["counts"])[:, None]).cuda()
    assert torch.equal(acc[held], twice[held]) and torch.equal(acc[~held], w.cuda()[~held])
    # decay 0 reads no weights
    out = torch.zeros_like(acc)
    v4a.v4a_attend_weights(q, own, l, None, out, decay=0.0, **kw)
    want = weights_call(v4a, c, lse, torch.full_like(w, math.nan), 0.0)
    assert torch.equal(out[held], want[held]) and torch.isfinite(out).all()


@pytest.mark.parametrize("dtype,H,d", [(F32, 4, 128), (BF16, 64, 512)])
def test_attend_weights_reports_bad_lengths(v4a, dtype, H, d):
    c = shared_case(dtype, 2, 1, H, d, 4, 10, 0, seed=16)
    w, lse = torch.zeros((2, 10)), torch.zeros((2, 1, H))
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    weights_call(v4a, c, lse, w, 1.0, dev_status=status)
    assert int(status) == 0
    c["lens"][1] = -5
    out = weights_call(v4a, c, lse, w, 1.0, dev_status=status)
    assert int(status) == 4 and (out[1, : c["counts"][1]] == 0).all()


# ------------------------------------------------------------------ eviction

EVICT = [
    # dtype, B, rows, d, budget, first, recent, out_rows
    (BF16, 2, 100, 512, 40, 4, 8, 40), (F32, 3, 33, 64, 33, 0, 0, 50), (F32, 1, 1, 4, 1, 0, 0, 1), (BF16, 1, 2500, 64, 7, 3, 4, 7),
    (BF16, 4, 1024, 8, 1000, 0, 100, 1000), (F32, 2, 9000, 12, 4097, 1, 1, 4100), (BF16, 1, 70000, 8, 1, 0, 0, 2), (F32, 2, 5, 64, 20, 2, 2, 20)]


def evict_case(dtype, B, rows, d, seed, ragged=True, kind="ties"):
    g = gen(seed)
    own = normal(g, (B, rows, d), dtype)
    w = torch.randn((B, rows), generator=g)
    if kind == "ties":
        w = (w * 2).round() / 2
        w[torch.rand((B, rows), generator=g) < 0.2] = 0.0
        w[torch.rand((B, rows), generator=g) < 0.05] = -0.0
    if kind == "equal":
        w = torch.ones((B, rows))
    if kind == "special":
        for v in (math.inf, -math.inf, math.nan, 1e-42, -1e-42, 3.4e38):
            w[torch.rand((B, rows), generator=g) < 0.1] = v
    counts = [int(torch.randint(0, rows + 1, (1,), generator=g)) if ragged and b else rows for b in range(B)]
    return own, w, counts


@pytest.mark.parametrize("dtype,B,rows,d,budget,first,recent,out_rows", EVICT)
@pytest.mark.parametrize("kind", ["ties", "equal", "special", "spread"])
def test_evict(v4a, dtype, B, rows, d, budget, first, recent, out_rows, kind):
    own, w, counts = evict_case(dtype, B, rows, d, seed=17, kind=kind)
    entries = torch.randint(1, 3, (B, rows), generator=gen(18)).cumsum(1).to(torch.int32)
    want = su.evict_ref(w, counts, budget, first, recent)
    o = dict(own=torch.full((B, out_rows, d), 7.0, dtype=dtype, device="cuda"), w=torch.full((B, out_rows), 7.0, device="cuda"),
             kept=torch.full((B, budget), 7, dtype=torch.int32, device="cuda"), n=torch.full((B,), 7, dtype=torch.int32, device="cuda"),
             e=torch.full((B, out_rows), 7, dtype=torch.int32, device="cuda"))
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    for with_entries in (True, False):
        v4a.v4a_evict(own.cuda(), w.cuda(), o["own"], o["w"], o["kept"], o["n"], budget=budget, keep_first=first, keep_recent=recent,
                      own_count=torch.tensor(counts, dtype=torch.int32).cuda(), own_entry=entries.cuda() if with_entries else None,
                      entry_out=o["e"], first_entry=1000, dev_status=status)
        assert int(status) == 0
        h = {k: t.cpu() for k, t in o.items()}
        for b, keep in enumerate(want):
            n = len(keep)
            assert int(h["n"][b]) == n
            assert h["kept"][b].tolist() == keep + [-1] * (budget - n)
            assert torch.equal(h["own"][b, :n], own[b, keep])
            assert torch.equal(h["w"][b, :n].view(torch.int32), w[b, keep].view(torch.int32))  # to the bit, NaN and -0 too
            e = entries[b, keep] if with_entries else torch.tensor(keep, dtype=torch.int32) + 1000
            assert torch.equal(h["e"][b, :n], e)
            # behind the kept ones: as it was
            assert (h["own"][b, n:] == 7).all() and (h["w"][b, n:] == 7).all() and (h["e"][b, n:] == 7).all()


def test_evict_without_counts_and_bad_counts(v4a):
    own, w, _ = evict_case(F32, 2, 50, 8, seed=19, ragged=False)
    own, w = own.cuda(), w.cuda()

    def call(**kw):
        o = [torch.zeros((2, 10, 8), device="cuda"), torch.zeros((2, 10), device="cuda"),
             torch.zeros((2, 10), dtype=torch.int32, device="cuda"), torch.zeros((2,), dtype=torch.int32, device="cuda")]
        v4a.v4a_evict(own, w, *o, budget=10, keep_first=1, keep_recent=2, **kw)
        return o

    want = su.evict_ref(w.cpu(), [50, 50], 10, 1, 2)
    assert call()[2].tolist() == want
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    o = call(own_count=torch.tensor([-4, 51], dtype=torch.int32, device="cuda"), dev_status=status)
    assert int(status) == 4
    assert o[2].tolist() == [[-1] * 10, want[1]] and o[3].tolist() == [0, 10]


def test_evict_captured(v4a):
    own, w, counts = evict_case(BF16, 3, 3000, 64, seed=20)
    own, w, cnt = own.cuda(), w.cuda(), torch.tensor(counts, dtype=torch.int32).cuda()
    o = [torch.zeros((3, 500, 64), dtype=BF16, device="cuda"), torch.zeros((3, 500), device="cuda"),
         torch.zeros((3, 500), dtype=torch.int32, device="cuda"), torch.zeros((3,), dtype=torch.int32, device="cuda")]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v4a.v4a_evict(own, w, *o, budget=500, keep_first=4, keep_recent=32, own_count=cnt)
    for seed in (21, 22):
        w.copy_(torch.randn(w.shape, generator=gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        for b, keep in enumerate(su.evict_ref(w.cpu(), counts, 500, 4, 32)):
            assert o[2][b].tolist() == keep + [-1] * (500 - len(keep))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,H,d", [(F32, 8, 128), (BF16, 64, 512)])
def test_serving_steps_together(v4a, dtype, H, d):
    """Decode steps of a batch behind a shared prefix, as a serving program runs them: rotate the new rows, append to the
    ring, compress a completed chunk into the next own slot, attend, add up the weights, and evict when the cache is
    full -- against the plain forms fed with the library's own rotated rows and entries."""
    g = gen(30)
    B, m, W, Np, cap, budget, ring_rows = 2, 8, 16, 12, 6, 3, 32
    prefix = normal(g, (Np, d), dtype).cuda()
    ring, gate_ring = torch.zeros((B, ring_rows, d), dtype=dtype, device="cuda"), torch.zeros((B, ring_rows, d), dtype=dtype, device="cuda")
    own = torch.full((B, cap, d), math.nan, dtype=dtype, device="cuda")
    spare, entry, spare_e = own.clone(), torch.full((B, cap), -1, dtype=torch.int32, device="cuda"), torch.zeros((B, cap), dtype=torch.int32, device="cuda")
    acc, spare_w = torch.zeros((B, cap), device="cuda"), torch.zeros((B, cap), device="cuda")
    count = torch.zeros((B,), dtype=torch.int32, device="cuda")
    kept = torch.zeros((B, budget), dtype=torch.int32, device="cuda")
    n, evictions, total = 0, 0, 0  # own entries in the cache, evictions, own entries so far
    sums = torch.zeros((B, cap), dtype=torch.float64)
    slack = torch.zeros((B, cap), dtype=torch.float64)
    for pos in range(m * Np, m * Np + 80):
        q, kv, gate = (normal(g, s, dtype).cuda() for s in ((B, 1, H, d), (B, 1, d), (B, d)))
        v4a.v4a_rope([(q, q), (kv, kv)], rope_dims=64, pos0=pos)
        v4a.v4a_ring_append([(kv[:, 0], ring), (gate, gate_ring)], pos)
        L = pos + 1
        if L % m == 0:  # a chunk is complete: the newest entry goes to slot n
            at = (L - m) % ring_rows
            v4a.v4a_compress(ring[:, at:], gate_ring[:, at:], own[:, n:], m=m, n_tok=m)
            entry[:, n] = Np + total
            acc[:, n] = 0
            n, total = n + 1, total + 1
            count.fill_(n)
        out, lse = torch.empty_like(q), torch.empty((B, 1, H), device="cuda")
        v4a.v4a_hca_attend_shared(q, prefix, own, ring, out, m=m, window=W, ctx_len=L, own_count=count, own_entry=entry, lse=lse, rope_dims=64)
        v4a.v4a_attend_weights(q, own, lse, acc, acc, m=m, ctx_len=L, n_prefix=Np, own_count=count, own_entry=entry)
        if L % m == 0 or pos % 17 == 0:
            host = dict(lens=[L] * B, counts=[n] * B, entries=entry.tolist(), m=m)
            bf = dtype == BF16
            ref, rl, tol, tol_l = su.shared_ref(q.cpu(), prefix.cpu(), own.cpu(), ring.cpu(), W=W, rope_dims=64, p_rounding=su.BF if bf else su.U,
                                                out_rounding=su.BF if bf else su.U, **host)
            within(out, ref, tol, f"out at {pos}")
            within(lse, rl, tol_l, f"lse at {pos}")
        got, tw = su.weights_ref(q.cpu(), own.cpu(), lse.cpu(), sums, n_prefix=Np, lens=[L] * B, counts=[n] * B, entries=entry.tolist(), m=m, decay=1.0)
        slack[:, :n] += tw[:, :n] + got[:, :n] * su.U
        sums[:, :n] = got[:, :n]
        within(acc[:, :n], sums[:, :n], slack[:, :n] + 1e-30, f"weights at {pos}")
        if n == cap:
            want = su.evict_ref(acc.cpu(), [n] * B, budget, 1, 1)
            v4a.v4a_evict(own, acc, spare, spare_w, kept, count, budget=budget, keep_first=1, keep_recent=1, own_entry=entry, entry_out=spare_e)
            assert kept.tolist() == want
            own, spare, acc, spare_w, entry, spare_e = spare, own, spare_w, acc, spare_e, entry
            k = torch.tensor(want)
            sums[:, :budget], slack[:, :budget] = sums.gather(1, k), slack.gather(1, k)
            sums[:, budget:], slack[:, budget:] = 0, 0
            n, evictions = budget, evictions + 1
    assert evictions >= 2
