"""The serving operators at their limits: sizes that take a kernel's other branches, sinks that outweigh every key, waits
that run out, workspaces made for another stream."""
import ctypes
import math

import pytest
import torch

import serving_utils as su
from test_gpu_serving import BF16, F32, attend, check_shared, evict_case, gen, normal, shared_case, weights_call, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def v4a():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import compressed_sparse_long_v4a_b200 as v
    return v


# ------------------------------------------------------------------ shared-prefix attention

@pytest.mark.parametrize("dtype,H,d", [(F32, 4, 128), (BF16, 64, 512), (BF16, 8, 512), (BF16, 4, 128)])
@pytest.mark.parametrize("size", [60.0, 300.0, 3e4])
def test_sink_that_outweighs_every_key(v4a, dtype, H, d, size):
    # e^(sink - the largest logit) overflows fp32 from about 88 on; the denominator's logarithm is the sink then
    c = shared_case(dtype, 2, 1, H, d, 60, 5, 16, seed=40)
    sink = torch.full((H,), size)
    sink[0] = -size  # and one that weighs nothing
    check_shared(v4a, c, sink=sink)


@pytest.mark.parametrize("dtype,T,H,d,Np,rows,W", [(F32, 90, 2, 64, 10, 40, 20), (BF16, 150, 2, 512, 10, 40, 20), (BF16, 70, 3, 512, 0, 3, 300),
                                                   (BF16, 300, 1, 512, 3, 0, 1)])
@pytest.mark.parametrize("slack", [0, 40])
def test_many_queries_of_a_sequence(v4a, dtype, T, H, d, Np, rows, W, slack):
    # their windows together are longer than a tile, and wrap around the ring's end
    check_shared(v4a, shared_case(dtype, 2, T, H, d, Np, rows, W, m=64, seed=41, ring_rows=W + T - 1 + slack))


@pytest.mark.parametrize("Np", [63, 64, 65, 127, 128, 129, 255, 257, 1000])
def test_prefix_lengths_around_the_tiles(v4a, Np):
    check_shared(v4a, shared_case(BF16, 3, 1, 24, 512, Np, 2, 3, seed=42))


@pytest.mark.parametrize("W,ring_rows,at", [(64, 64, 0), (128, 128, 1), (128, 191, 190), (127, 130, 64), (129, 129, 128), (1, 1, 0)])
def test_windows_that_wrap_anywhere(v4a, W, ring_rows, at):
    c = shared_case(BF16, 2, 1, 64, 512, 0, 0, W, seed=43, ring_rows=ring_rows)
    c["lens"] = [7 * ring_rows + at + 1, 3 * ring_rows + (at + 50) % ring_rows + 1]
    c["ctx_len"] = max(c["lens"])
    check_shared(v4a, c)


def test_more_groups_of_rows_than_pairs_can_have_pieces(v4a):
    # 76,800 rows are 600 groups of 128
    g = gen(44)
    B, H, d, Np = 600, 128, 512, 3
    q, prefix = torch.randn((B, 1, H, d), generator=g).to(BF16), normal(g, (Np, d), BF16)
    out, lse = torch.zeros((B, 1, H, d), dtype=BF16, device="cuda"), torch.zeros((B, 1, H), device="cuda")
    v4a.v4a_hca_attend_shared(q.cuda(), prefix.cuda(), None, None, out, m=1, window=0, ctx_len=Np, lse=lse)
    s = q.double() @ prefix.double().T / math.sqrt(d)
    z = torch.logsumexp(s, -1)
    ref = (s - z[..., None]).exp() @ prefix.double()
    e = ((d + 2) * su.U * q.double().norm(dim=-1, keepdim=True) * prefix.double().norm(dim=1) / math.sqrt(d) + 4 * su.U * s.abs()).amax(-1)
    n = Np + 8
    within(lse, z, 1.01 * e + n * su.U + 4 * su.U * z.abs() + 4 * su.U, "lse")
    tol = ((s - z[..., None]).exp() @ prefix.double().abs()) * (2.02 * e + n * 2 * su.U + su.BF)[..., None]
    within(out, ref, tol + ref.abs() * su.BF, "out")


def test_maxima_that_keep_growing(v4a):
    # every tile's largest logit is far above the one before: the output so far is scaled down again and again
    c = shared_case(BF16, 1, 1, 64, 512, 1100, 1, 0, seed=45)
    c["prefix"] = (c["prefix"].float() * torch.linspace(0.05, 12.0, 1100)[:, None]).to(BF16)
    check_shared(v4a, c)
    c["prefix"] = c["prefix"].flip(0).contiguous()
    check_shared(v4a, c)


def test_infinities_in_visible_entries_stay_in_their_sequence(v4a):
    c = shared_case(BF16, 4, 1, 32, 512, 70, 40, 16, ragged=False, seed=46)
    clean, lse = attend(v4a, c)
    for bad in (math.inf, -math.inf):
        for key, at in (("own", (2, 7)), ("own", (2, 7, 300)), ("ring", (2,))):
            d2 = {**c, key: c[key].clone()}
            d2[key][at] = bad
            out, l2 = attend(v4a, d2)
            others = [0, 1, 3]
            assert torch.equal(out[others], clean[others]) and torch.equal(l2[others], lse[others])


@pytest.mark.parametrize("tile", [0, 1])
def test_waits_that_run_out(v4a, tile):
    c = shared_case(BF16, 8, 1, 64, 512, 8192, 70, 128, seed=47)
    good, lse = attend(v4a, c)
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    v4a.lib.v4a_test_attend_fault(ctypes.c_int(tile), ctypes.c_int(64))
    try:
        out, l = attend(v4a, c, status=status)
        torch.cuda.synchronize()
    finally:
        v4a.lib.v4a_test_attend_fault(ctypes.c_int(-1), ctypes.c_int(0))
    assert int(status) == 4
    assert torch.isnan(out).flatten(1).any(1).all()  # each group of rows has a pair that gave up
    again, l = attend(v4a, c, status=status)
    assert int(status) == 0 and torch.equal(again, good) and torch.equal(l, lse)


def test_workspace_of_the_call_on_another_stream(v4a):
    # no workspace given: the call's own one is used on a stream that is not the current one
    c = shared_case(BF16, 16, 1, 64, 512, 4096, 70, 128, seed=48)
    want, _ = attend(v4a, c)
    dev = {k: c[k].cuda() for k in ("q", "prefix", "own", "ring")}
    lens, cnt = torch.tensor(c["lens"]).cuda(), torch.tensor(c["counts"], dtype=torch.int32).cuda()
    out = torch.empty_like(dev["q"])
    size = v4a.v4a_shared_workspace_size(batch=16, heads=64, d=512, n_prefix=4096, own_rows=70, window=128)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        for stream in (side, side.cuda_stream):
            v4a.v4a_hca_attend_shared(dev["q"], dev["prefix"], dev["own"], dev["ring"], out, m=128, window=128, ctx_len=c["ctx_len"],
                                      ctx_lens=lens, own_count=cnt, stream=stream)
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)  # what the current stream gets next
        side.synchronize()
        assert torch.equal(out, want)
        torch.cuda.synchronize()


@pytest.mark.parametrize("raw", [False, True])
def test_workspace_of_the_call_takes_no_memory_that_the_current_stream_still_uses(v4a, raw):
    # a temporary of the current stream, let go of while kernels that read it are queued: its block may serve that stream
    # again at once, but no other
    c = shared_case(BF16, 16, 1, 64, 512, 4096, 70, 128, seed=59)
    want, _ = attend(v4a, c)
    dev = {k: c[k].cuda() for k in ("q", "prefix", "own", "ring")}
    lens, cnt = torch.tensor(c["lens"]).cuda(), torch.tensor(c["counts"], dtype=torch.int32).cuda()
    out = torch.empty_like(dev["q"])
    size = v4a.v4a_shared_workspace_size(batch=16, heads=64, d=512, n_prefix=4096, own_rows=70, window=128)
    copy = torch.empty(size, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        tmp = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(20_000_000)  # 10 ms: the call below is done long before
        copy.copy_(tmp)
        del tmp
        v4a.v4a_hca_attend_shared(dev["q"], dev["prefix"], dev["own"], dev["ring"], out, m=128, window=128, ctx_len=c["ctx_len"],
                                  ctx_lens=lens, own_count=cnt, stream=side.cuda_stream if raw else side)
        side.synchronize()
        assert torch.equal(out, want)
        assert (copy == 7).all()


def test_capture_on_another_stream_needs_a_workspace(v4a):
    # the call's own workspace would go back to the allocator, and the graph would keep writing to it
    q, prefix = torch.randn((2, 1, 4, 128), device="cuda"), torch.randn((50, 128), device="cuda")
    out, want = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(v4a.v4a_shared_workspace_size(batch=2, heads=4, d=128, n_prefix=50, own_rows=0, dtype=F32), dtype=torch.uint8, device="cuda")
    kw = dict(m=128, window=0, ctx_len=128 * 50)
    v4a.v4a_hca_attend_shared(q, prefix, None, None, want, **kw)
    torch.cuda.synchronize()
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            with pytest.raises(ValueError, match="workspace"):
                v4a.v4a_hca_attend_shared(q, prefix, None, None, out, stream=side, **kw)
            v4a.v4a_hca_attend_shared(q, prefix, None, None, out, workspace=ws, stream=side, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("d,H", [(512, 64), (512, 8), (256, 128)])
def test_output_as_the_next_calls_query(v4a, d, H):
    # the attention kernels request their first query early: it must be the output of the call before, call after call
    g = gen(49)
    T = 512 // d * 64 // H if d * H < 32768 else 1  # [2][1][64][512] in all
    prefix, ent = normal(g, (300, d), BF16).cuda(), normal(g, (2, 700, 512), BF16).cuda()
    ring = torch.zeros((2, 1, 512), dtype=BF16, device="cuda")
    qs = [normal(g, (2, T, H, d), BF16).cuda() for _ in range(6)]
    mid, want, got = torch.empty_like(qs[0]), [], []

    def step(q, wait):
        v4a.v4a_hca_attend_shared(q, prefix, None, None, mid, m=128, window=0, ctx_len=128 * 300 + T)
        if wait:
            torch.cuda.synchronize()
        o = torch.empty((2, 1, 64, 512), device="cuda")
        v4a.v4a_hca_attend(mid.view(2, 1, 64, 512), ent, ring, 700 * 128 - 1, o, m=128, window=0, ctx_len=700 * 128)
        return o

    for q in qs:
        want.append(step(q, True))
        torch.cuda.synchronize()
    for _ in range(20):
        got = [step(q, False) for q in qs]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("dtype,H,d", [(F32, 3, 64), (BF16, 3, 64), (BF16, 20, 512)])
def test_weights_of_many_short_sequences(v4a, dtype, H, d):
    # more sequences than a block has threads; many of them empty
    c = shared_case(dtype, 700, 1, H, d, 1, 3, 0, seed=50)
    g = gen(51)
    w, lse = torch.rand((700, 3), generator=g), torch.randn((700, 1, H), generator=g) + 2
    ref, tol = su.weights_ref(c["q"], c["own"], lse, w, n_prefix=1, lens=c["lens"], counts=c["counts"], entries=None, m=128, decay=0.5)
    out = weights_call(v4a, c, lse, w, 0.5)
    held = ~torch.isnan(ref)
    assert (out.cpu()[~held] == 7.0).all()
    within(torch.where(held.cuda(), out, 0.0), torch.where(held, ref, 0.0), tol, "weights")


@pytest.mark.parametrize("dtype,T,H,d,rows", [(BF16, 1, 15, 128, 1000), (BF16, 9, 64, 256, 130), (BF16, 2, 128, 512, 700), (F32, 11, 9, 64, 70)])
def test_weights_of_long_caches_and_many_rows(v4a, dtype, T, H, d, rows):
    c = shared_case(dtype, 3, T, H, d, 0, rows, 0, seed=52, evicted=True)
    q, own = c["q"].cuda().double(), c["own"].cuda().double()
    g = gen(53)
    lse = torch.randn((3, T, H), generator=g) + 4
    w = torch.rand((3, rows), generator=g)
    s = torch.einsum("bthd,bnd->bthn", q, own) / math.sqrt(d)
    t = torch.tensor(su.query_positions(c["lens"], T)).cuda()
    e = torch.tensor(c["entries"]).cuda()
    seen = 128 * (e[:, None] + 1) <= t[:, :, None] + 1
    p = (s - lse.cuda().double()[..., None]).exp() * seen[:, :, None]
    ref = w.cuda().double() + p.sum((1, 2))
    eps = (d + 2) * su.U * q.norm(dim=-1)[..., None] * own.norm(dim=-1)[:, None, None] / math.sqrt(d) + 4 * su.U * (s.abs() + lse.cuda().abs()[..., None])
    tol = (p * (1.02 * eps + (T * H + 8) * su.U)).sum((1, 2)) + ref * 2 * su.U
    held = torch.arange(rows) < torch.tensor(c["counts"])[:, None]
    out = weights_call(v4a, c, lse, w, 1.0)
    within(torch.where(held.cuda(), out, 0.0), torch.where(held, ref.cpu(), 0.0), tol.cpu(), "weights")
    assert (out.cpu()[~held] == 7.0).all()


# ------------------------------------------------------------------ eviction

@pytest.mark.parametrize("rows,budget", [(800_000, 300_000), (140_001, 70_001), (66_000, 5)])
@pytest.mark.parametrize("kind", ["ties", "equal", "special", "spread"])
def test_evict_very_long(v4a, rows, budget, kind):
    # clusters of 16 blocks; the longest does not fit their shared memory
    own, w, _ = evict_case(BF16, 1, rows, 8, seed=54, ragged=False, kind=kind)
    o = [torch.zeros((1, budget, 8), dtype=BF16, device="cuda"), torch.zeros((1, budget), device="cuda"),
         torch.zeros((1, budget), dtype=torch.int32, device="cuda"), torch.zeros((1,), dtype=torch.int32, device="cuda")]
    v4a.v4a_evict(own.cuda(), w.cuda(), *o, budget=budget, keep_first=2, keep_recent=3)
    key = w[0].double()
    key[torch.isnan(w[0])] = -math.inf  # last; the infinities among the weights have room before them
    key[w[0] == -math.inf], key[w[0] == math.inf] = -1e300, 1e300
    key[:2] = key[-3:] = math.inf
    want = key.argsort(descending=True, stable=True)[:budget].sort().values
    assert torch.equal(o[2][0].cpu().long(), want) and int(o[3]) == budget
    assert torch.equal(o[0][0].cpu(), own[0, want]) and torch.equal(o[1][0].cpu().view(torch.int32), w[0, want].view(torch.int32))


def test_evict_very_long_captured(v4a):
    own, w, _ = evict_case(BF16, 1, 100_000, 8, seed=55, ragged=False, kind="spread")
    own, w = own.cuda(), w.cuda()
    o = [torch.zeros((1, 400, 8), dtype=BF16, device="cuda"), torch.zeros((1, 400), device="cuda"),
         torch.zeros((1, 400), dtype=torch.int32, device="cuda"), torch.zeros((1,), dtype=torch.int32, device="cuda")]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v4a.v4a_evict(own, w, *o, budget=400)
    w.copy_(torch.randn(w.shape, generator=gen(56)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o[2][0].long(), w[0].argsort(descending=True, stable=True)[:400].sort().values)


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("dtype,B,T,H,d,R", [(F32, 3, 333, 1, 64, 16), (BF16, 2, 500, 2, 128, 64), (F32, 2, 301, 5, 128, 128), (BF16, 1, 40, 1, 4096, 512),
                                             (BF16, 5, 200, 4, 512, 64), (F32, 1, 900, 3, 24, 16)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_tokens_of_few_rows(v4a, dtype, B, T, H, d, R, half, in_place):
    # several tokens share a block, across the ends of sequences; rows of 512 items
    g = gen(57)
    x = normal(g, (B, T, H, d), dtype)
    pos = torch.randint(0, 1 << 20, (B, T), generator=g)
    dx = x.cuda()
    out = dx if in_place else torch.full_like(dx, 7.0)
    v4a.v4a_rope([(dx, out)], rope_dims=R, positions=pos.cuda(), half=half)
    ref = su.rope_ref(x, pos, R, d - R, half)
    within(out, ref, su.rope_bound(x, ref, pos, R, d - R, rounding=su.BF if dtype == BF16 else su.U), "rope")
    assert torch.equal(out.cpu()[..., : d - R], x[..., : d - R])


@pytest.mark.parametrize("dtype,B,T,H,d,R", [(BF16, 3, 333, 7, 512, 64), (F32, 2, 700, 31, 64, 32), (BF16, 1, 2500, 5, 256, 128), (BF16, 1, 12000, 1, 128, 32)])
@pytest.mark.parametrize("half,in_place", [(False, False), (False, True), (True, False), (True, True)])
def test_rope_blocks_of_several_tokens(v4a, dtype, B, T, H, d, R, half, in_place):
    # enough tokens that a block takes several, with more rows than it has threads for; beside them one-head rows between
    # others' rows, left as they were
    g = gen(58)
    x, kv = normal(g, (B, T, H, d), dtype), normal(g, (B, T, 3, d), dtype)
    pos = torch.randint(0, 1 << 20, (B, T), generator=g)
    dx, dkv = x.cuda(), kv.cuda()
    out = dx if in_place else torch.full_like(dx, 7.0)
    v4a.v4a_rope([(dx, out), (dkv[:, :, 1], dkv[:, :, 1])], rope_dims=R, positions=pos.cuda(), half=half, rope_offset=0)
    rounding = su.BF if dtype == BF16 else su.U
    for a, b in ((x, out), (kv[:, :, 1:2], dkv[:, :, 1:2])):
        ref = su.rope_ref(a, pos, R, 0, half)
        within(b, ref, su.rope_bound(a, ref, pos, R, 0, rounding=rounding), "rope")
        assert torch.equal(b.cpu()[..., R:], a[..., R:])
    assert torch.equal(dkv[:, :, ::2].cpu(), kv[:, :, ::2])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rope_streams_between_each_others_rows(v4a, dtype):
    # one fused tensor: two parts of the same rows in place, heads in place, and heads written over others that nobody reads
    g = gen(62)
    fused = normal(g, (2, 5, 9, 256), dtype)
    pos = torch.randint(0, 1 << 20, (2, 5), generator=g)
    f = fused.cuda()
    v4a.v4a_rope([(f[:, :, 0:2], f[:, :, 0:2]), (f[:, :, 0:2, :128], f[:, :, 0:2, :128]), (f[:, :, 2], f[:, :, 2]), (f[:, :, 3:6], f[:, :, 6:9])],
                 rope_dims=64, positions=pos.cuda())
    rounding = su.BF if dtype == BF16 else su.U

    def check(got, x, off):
        ref = su.rope_ref(x, pos, 64, off)
        within(got[..., off : off + 64], ref[..., off : off + 64], su.rope_bound(x, ref, pos, 64, off, rounding=rounding)[..., off : off + 64], "rope")

    check(f[:, :, 0:3], fused[:, :, 0:3], 192)
    check(f[:, :, 0:2], fused[:, :, 0:2], 64)
    check(f[:, :, 6:9], fused[:, :, 3:6], 192)
    f = f.cpu()
    assert torch.equal(f[:, :, 3:6], fused[:, :, 3:6]) and torch.equal(f[:, :, 6:9, :192], fused[:, :, 3:6, :192])
    assert torch.equal(f[:, :, 0:2, :64], fused[:, :, 0:2, :64]) and torch.equal(f[:, :, 0:2, 128:192], fused[:, :, 0:2, 128:192])
    assert torch.equal(f[:, :, 2, :192], fused[:, :, 2, :192])


def test_rope_refuses_an_out_shifted_against_its_x(v4a):
    x = torch.zeros((1, 9, 4, 64), device="cuda")
    with pytest.raises(v4a.V4AError, match="overlap"):
        v4a.v4a_rope([(x[:, :8], x[:, 1:])], rope_dims=64)
    with pytest.raises(v4a.V4AError, match="overlap"):
        v4a.v4a_rope([(x[:, :4], x[:, 4:8]), (x[:, 5:9], x[:, 5:9])], rope_dims=64)
