"""What the serving calls refuse, found on the host before anything is launched (no GPU needed): the pointers
below are never dereferenced."""
import ctypes

import pytest

FAKE = 1 << 20
INVALID, UNSUPPORTED, OK = 1, 2, 0


@pytest.fixture(scope="module")
def v4a():
    import compressed_sparse_long_v4a_b200 as v
    return v


def rope_io(v, **kw):
    f = dict(x=FAKE, out=2 * FAKE, heads=4, d=64, rope_offset=0, dtype=1, x_batch_stride=1024, x_tok_stride=256,
             x_head_stride=64, out_batch_stride=1024, out_tok_stride=256, out_head_stride=64)
    f.update(kw)
    return v.RopeIO(**f)


def rope(v, io=None, n=1, batch=2, n_tok=4, positions=None, pos_stride=0, **kw):
    f = dict(rope_dims=64, half=0, inverse=0, base=10000.0, factor=1.0, orig_ctx=0, beta_fast=32.0, beta_slow=1.0,
             out_scale=1.0)
    f.update(kw)
    p = v.RopeParams(**f)
    arr = (v.RopeIO * 9)()
    for i in range(9):
        arr[i] = io if io is not None else rope_io(v)
    return v.lib.v4a_rope(arr, n, batch, n_tok, positions, pos_stride, 0, 1, ctypes.byref(p), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rope_dims=63), INVALID), (dict(rope_dims=0), INVALID), (dict(rope_dims=514), INVALID), (dict(base=0.0), INVALID),
    (dict(factor=0.0), INVALID), (dict(factor=float("nan")), INVALID), (dict(orig_ctx=-1), INVALID),
    (dict(orig_ctx=4096, beta_fast=1.0), INVALID), (dict(out_scale=float("inf")), INVALID), (dict(n=9), INVALID),
    (dict(n=-1), INVALID), (dict(batch=-1), INVALID), (dict(n_tok=-1), INVALID), (dict(positions=FAKE + 4), INVALID),
    (dict(positions=FAKE, pos_stride=-1), INVALID), (dict(n_tok=1 << 31), UNSUPPORTED),
    (dict(n=0), OK), (dict(batch=0), OK), (dict(n_tok=0), OK)])
def test_rope_arguments(v4a, kw, status):
    assert rope(v4a, **kw) == status
    if status:
        assert b"v4a_rope" in v4a.lib.v4a_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(heads=0), INVALID), (dict(d=62), INVALID),
    (dict(rope_offset=1), INVALID), (dict(rope_offset=-1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(x=FAKE + 1), INVALID), (dict(x_tok_stride=-1), INVALID),
    # rows of out that overlap: a broadcast dimension, strides below the row, a batch inside the tokens
    (dict(out_head_stride=0), INVALID), (dict(out_tok_stride=0), INVALID), (dict(out_head_stride=63), INVALID),
    (dict(out_batch_stride=512), INVALID),
    # in place with other strides
    (dict(out=FAKE, out_tok_stride=512, out_batch_stride=2048), INVALID)])
def test_rope_streams(v4a, kw, status):
    assert rope(v4a, rope_io(v4a, **kw)) == status


def test_rope_streams_share_a_dtype(v4a):
    p = v4a.RopeParams(64, 0, 0, 10000.0, 1.0, 0, 32.0, 1.0, 1.0)
    arr = (v4a.RopeIO * 2)(rope_io(v4a), rope_io(v4a, dtype=0))
    assert v4a.lib.v4a_rope(arr, 2, 2, 4, None, 0, 0, 1, ctypes.byref(p), None) == UNSUPPORTED
    assert v4a.lib.v4a_rope(None, 1, 2, 4, None, 0, 0, 1, ctypes.byref(p), None) == INVALID
    assert v4a.lib.v4a_rope(arr, 1, 2, 4, None, 0, 0, 1, None, None) == INVALID


@pytest.mark.parametrize("kw", [dict(beta_fast=float("inf")), dict(beta_slow=float("-inf")), dict(beta_slow=float("nan"))])
def test_rope_blend_without_bounds(v4a, kw):
    # the blend would be 0 * inf: every angle a NaN
    assert rope(v4a, orig_ctx=4096, n_tok=4, **kw) == INVALID
    assert rope(v4a, orig_ctx=0, n_tok=0, **kw) == OK  # not used


def test_rope_streams_that_write_over_each_other(v4a):
    # the same tensor twice would be turned twice, or half of it, as the blocks happen to run
    p = v4a.RopeParams(64, 0, 0, 10000.0, 1.0, 0, 32.0, 1.0, 1.0)
    far, call = 64 * FAKE, lambda *ios: v4a.lib.v4a_rope((v4a.RopeIO * len(ios))(*ios), len(ios), 2, 4, None, 0, 0, 1, ctypes.byref(p), None)
    one = rope_io(v4a)
    for x, out in ((one.x, one.out), (far, one.out), (one.out, far), (far, one.x)):
        assert call(one, rope_io(v4a, x=x, out=out)) == INVALID
        assert call(one, rope_io(v4a, x=3 * far, out=4 * far), rope_io(v4a, x=x, out=out)) == INVALID
    assert b"overlap" in v4a.lib.v4a_last_error()


# The overlap checks of v4a_rope.  A last stream of another dtype is refused for that (UNSUPPORTED) once all others have
# been accepted, so nothing is ever launched.
def rope_overlap(v4a, ios, batch, n_tok, rope_dims):
    p = v4a.RopeParams(rope_dims, 0, 0, 10000.0, 1.0, 0, 32.0, 1.0, 1.0)
    arr = (v4a.RopeIO * (len(ios) + 1))(*ios, rope_io(v4a, dtype=3))
    status = v4a.lib.v4a_rope(arr, len(ios) + 1, batch, n_tok, None, 0, 0, 1, ctypes.byref(p), None)
    if status == UNSUPPORTED:
        return False
    assert status == INVALID and b"overlap" in v4a.lib.v4a_last_error() and b"rows of out" not in v4a.lib.v4a_last_error()
    return True


@pytest.mark.parametrize("shift", [2, 64, 128, 512, 1024, 2 * (1024 + 256) - 2])
@pytest.mark.parametrize("back", [False, True])
def test_rope_out_that_overlaps_its_own_x_in_part(v4a, shift, back):
    # [2][4][4][64] bf16 with rows of one token 512 bytes, of one sequence 2,048 bytes apart: by elements, rows, tokens
    io = rope_io(v4a, x=8 * FAKE, out=8 * FAKE + (-shift if back else shift))
    assert rope_overlap(v4a, [io], 2, 4, 64)


def test_rope_rows_between_those_of_others(v4a):
    # heads of one fused projection [2][4][9][64]: in place, and from one part of it to another
    s = dict(x_batch_stride=4 * 576, x_tok_stride=576, x_head_stride=64, out_batch_stride=4 * 576, out_tok_stride=576, out_head_stride=64)
    at = lambda h: FAKE + 128 * h
    heads = lambda x, out, n: rope_io(v4a, x=at(x), out=at(out), heads=n, **s)
    assert not rope_overlap(v4a, [heads(0, 0, 4), heads(4, 4, 4), heads(8, 8, 1)], 2, 4, 64)
    assert not rope_overlap(v4a, [heads(0, 4, 4), heads(8, 8, 1)], 2, 4, 64)
    assert rope_overlap(v4a, [heads(0, 4, 5)], 2, 4, 64)  # its last head is the first of the outputs
    assert rope_overlap(v4a, [heads(0, 0, 4), heads(3, 3, 4)], 2, 4, 64)
    assert rope_overlap(v4a, [heads(0, 0, 4), heads(8, 4, 1), heads(4, 4, 1)], 2, 4, 64)
    # in place, two parts of the same rows: only the rotated dims count
    part = lambda off: rope_io(v4a, x=FAKE, out=FAKE, rope_offset=off)
    assert not rope_overlap(v4a, [part(0), part(32)], 2, 4, 32)
    assert rope_overlap(v4a, [part(0), part(30)], 2, 4, 32)


def test_rope_overlap_agrees_with_counting(v4a):
    import itertools
    import random
    rng = random.Random(1)
    seen = [0, 0]

    def layout(n, d):  # strides (batch, token, head) in elements that keep rows apart
        order, reach, s = rng.sample(range(3), 3), d, [0, 0, 0]
        for k in order:
            s[k] = reach + rng.choice([0, 0, 1, d, 3 * d])
            reach += (n[k] - 1) * s[k]
        return s

    for _ in range(4000):
        B, T, R = rng.randint(1, 3), rng.randint(1, 4), 2 * rng.randint(1, 2)
        ios, touched = [], []
        common = None
        for _ in range(rng.randint(1, 2)):
            H, d = rng.randint(1, 3), R + rng.randint(0, 3)
            xs = layout((B, T, H), d)
            if common and rng.random() < 0.5:
                xs, H, d = common
            common = (xs, H, d)
            x = FAKE + 2 * rng.randint(0, 120)
            in_place = rng.random() < 0.5
            os_ = xs if in_place or rng.random() < 0.5 else layout((B, T, H), d)
            out, off = x if in_place else FAKE + 2 * rng.randint(0, 240), rng.randint(0, d - R)
            if not in_place and out == x:
                continue
            ios.append(rope_io(v4a, x=x, out=out, heads=H, d=d, rope_offset=off, x_batch_stride=xs[0], x_tok_stride=xs[1], x_head_stride=xs[2],
                               out_batch_stride=os_[0], out_tok_stride=os_[1], out_head_stride=os_[2]))
            dims = range(off, off + R) if in_place else range(d)
            cells = lambda at, s: {at // 2 + b * s[0] + t * s[1] + h * s[2] + e for b, t, h, e in itertools.product(range(B), range(T), range(H), dims)}
            touched.append((cells(x, xs), cells(out, os_), in_place))
        bad = any(not p and r & w for r, w, p in touched)
        for (r0, w0, _), (r1, w1, _) in itertools.combinations(touched, 2):
            bad = bad or bool(w0 & w1 or w0 & r1 or r0 & w1)
        assert rope_overlap(v4a, ios, B, T, R) == bad
        seen[bad] += 1
    assert min(seen) > 500


def test_rope_strides_that_pass_every_address(v4a):
    assert rope(v4a, rope_io(v4a, x_tok_stride=1 << 61)) == INVALID
    assert rope(v4a, rope_io(v4a, out_batch_stride=1 << 62)) == INVALID


def cache(v, **kw):
    f = dict(prefix=FAKE, n_prefix=8, own=FAKE, own_rows=16, own_count=FAKE, own_entry=None, ring=FAKE, ring_rows=256,
             ctx_lens=FAKE)
    f.update(kw)
    return v.SharedCache(**f)


def shape(v, **kw):
    f = dict(batch=2, n_q=1, heads=8, d=128, m=128, k=0, window=128, ctx_len=128 * 64)
    f.update(kw)
    return v.Shape(**f)


def attend(v, c=None, s=None, q=FAKE, out=FAKE, out_dtype=0, dtype=1, ws=FAKE, ws_bytes=1 << 40, status=None, ext=None,
           lse=FAKE):
    c, s = c or cache(v), s or shape(v)
    return v.lib.v4a_hca_attend_shared(q, ctypes.byref(c), out, out_dtype, lse, dtype, ws, ws_bytes, status,
                                       ctypes.byref(ext) if ext is not None else None, ctypes.byref(s), None)


@pytest.mark.parametrize("c,s,kw,status", [
    ({}, dict(d=96), {}, UNSUPPORTED), ({}, dict(heads=0), {}, INVALID), ({}, dict(n_q=0), {}, INVALID),
    ({}, dict(n_q=9, ctx_len=8), {}, INVALID), ({}, dict(batch=65536), {}, UNSUPPORTED), ({}, dict(m=0), {}, INVALID),
    ({}, dict(window=-1), {}, INVALID), ({}, dict(window=257), {}, INVALID), ({}, dict(window=256, n_q=2), {}, INVALID),
    (dict(ring=None), {}, {}, INVALID), (dict(n_prefix=65), {}, {}, INVALID), (dict(n_prefix=-1), {}, {}, INVALID),
    (dict(prefix=None), {}, {}, INVALID), (dict(own=None), {}, {}, INVALID), (dict(own_rows=-1), {}, {}, INVALID),
    (dict(own=FAKE + 8), {}, {}, INVALID), (dict(own_count=FAKE + 2), {}, {}, INVALID), (dict(ctx_lens=FAKE + 4), {}, {}, INVALID),
    ({}, {}, dict(q=None), INVALID), ({}, {}, dict(out=None), INVALID), ({}, {}, dict(out=FAKE + 4), INVALID),
    ({}, {}, dict(dtype=2), UNSUPPORTED), ({}, {}, dict(out_dtype=2), UNSUPPORTED), ({}, {}, dict(dtype=0, out_dtype=1), UNSUPPORTED),
    ({}, {}, dict(ws=None), INVALID), ({}, {}, dict(ws_bytes=64), INVALID), ({}, {}, dict(ws=FAKE + 16), INVALID),
    ({}, {}, dict(lse=FAKE + 2), INVALID), ({}, {}, dict(status=FAKE + 1), INVALID), ({}, dict(batch=0), {}, OK)])
def test_shared_attention(v4a, c, s, kw, status):
    assert attend(v4a, cache(v4a, **c), shape(v4a, **s), **kw) == status


def test_shared_attention_options(v4a):
    assert attend(v4a, ext=v4a.AttendExt(None, 3, 10000.0)) == INVALID
    assert attend(v4a, ext=v4a.AttendExt(None, 130, 10000.0)) == INVALID
    assert attend(v4a, ext=v4a.AttendExt(None, 64, 0.0)) == INVALID
    assert attend(v4a, ext=v4a.AttendExt(FAKE + 2, 0, 10000.0)) == INVALID


def test_shared_workspace_size(v4a):
    n = v4a.v4a_shared_workspace_size(batch=4, heads=64, d=512, n_prefix=512, own_rows=16, window=128)
    assert n > 4 * 64 * 512 * 4
    assert v4a.v4a_shared_workspace_size(batch=4, heads=64, d=512, n_prefix=-1, own_rows=16) == 0
    assert v4a.v4a_shared_workspace_size(batch=0, heads=64, d=512, n_prefix=1, own_rows=16) == 0


@pytest.mark.parametrize("kw", [dict(d=96), dict(d=448), dict(d=1024), dict(heads=1025), dict(batch=65536), dict(window=-1), dict(window=1 << 30),
                                dict(n_prefix=1 << 30), dict(own_rows=1 << 30), dict(dtype=2), dict(dtype=3), dict(n_q=0)])
def test_shared_workspace_size_is_0_for_what_the_call_rejects(v4a, kw):
    f = dict(batch=1, n_q=1, heads=8, d=128, window=0, n_prefix=8, own_rows=16, dtype=1)

    def both(**kw):
        a = {**f, **kw}
        s = shape(v4a, batch=a["batch"], n_q=a["n_q"], heads=a["heads"], d=a["d"], window=a["window"], m=1, ctx_len=1 << 40)
        c = cache(v4a, n_prefix=a["n_prefix"], own_rows=a["own_rows"], ring_rows=(1 << 31) - 1)
        size = v4a.lib.v4a_shared_workspace_size(ctypes.byref(s), a["n_prefix"], a["own_rows"], a["dtype"])
        return size, attend(v4a, c, s, dtype=a["dtype"], ws=None)

    assert both()[0] > 0  # and the call, without a workspace, refuses that
    size, status = both(**kw)
    assert size == 0 and status in (INVALID, UNSUPPORTED) and b"workspace" not in v4a.lib.v4a_last_error()


def test_shared_workspace_size_of_other_dtypes(v4a):
    import torch
    f = dict(batch=1, heads=8, d=128, n_prefix=8, own_rows=16)
    assert v4a.v4a_shared_workspace_size(**f, dtype=torch.float16) == 0
    assert v4a.v4a_shared_workspace_size(**f, dtype=torch.float32) > 0 and v4a.v4a_shared_workspace_size(**f) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(lse=None), INVALID), (dict(w_in=None), INVALID), (dict(w_out=None), INVALID), (dict(decay=-1.0), INVALID),
    (dict(decay=float("nan")), INVALID), (dict(w_out=FAKE + 2), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(batch=0), OK)])
def test_attend_weights(v4a, kw, status):
    f = dict(lse=FAKE, w_in=FAKE, w_out=FAKE, decay=1.0, dtype=1, batch=2)
    f.update(kw)
    c, s = cache(v4a), shape(v4a, batch=f["batch"])
    assert v4a.lib.v4a_attend_weights(FAKE, ctypes.byref(c), f["lse"], f["w_in"], f["w_out"], f["decay"], f["dtype"], None,
                                      ctypes.byref(s), None) == status


@pytest.mark.parametrize("by", [4, -4, 2 * 16 * 4 - 4, 4 - 2 * 16 * 4])
def test_attend_weights_that_overlap_in_part(v4a, by):
    # [2][16] weights, written while another block still reads them
    c, s = cache(v4a), shape(v4a)
    assert v4a.lib.v4a_attend_weights(FAKE, ctypes.byref(c), FAKE, 9 * FAKE, 9 * FAKE + by, 1.0, 1, None, ctypes.byref(s), None) == INVALID
    assert b"overlap" in v4a.lib.v4a_last_error()


def evict(v, batch=2, budget=8, first=1, recent=2, status=None, **kw):
    f = dict(own=FAKE, weights=2 * FAKE, own_count=None, own_entry=None, own_rows=32, d=64, dtype=1, own_out=3 * FAKE,
             weights_out=4 * FAKE, entry_out=5 * FAKE, kept=6 * FAKE, count_out=7 * FAKE, out_rows=8, first_entry=0)
    f.update(kw)
    io = v.EvictIO(**f)
    return v.lib.v4a_evict(ctypes.byref(io), batch, budget, first, recent, status, None)


@pytest.mark.parametrize("kw,status", [
    (dict(budget=0), INVALID), (dict(first=-1), INVALID), (dict(recent=8), INVALID), (dict(out_rows=7), INVALID),
    (dict(d=4), INVALID), (dict(d=0), INVALID), (dict(own_rows=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(own=None), INVALID), (dict(kept=None), INVALID), (dict(count_out=None), INVALID), (dict(own=FAKE + 8), INVALID),
    (dict(weights=FAKE + 2), INVALID), (dict(own_out=FAKE), INVALID), (dict(weights_out=2 * FAKE + 64), INVALID),
    (dict(entry_out=4 * FAKE), INVALID), (dict(own_out=FAKE - 16), INVALID), (dict(status=FAKE + 1), INVALID),
    (dict(batch=-1), INVALID), (dict(batch=65536), INVALID), (dict(batch=0), OK)])
def test_evict(v4a, kw, status):
    assert evict(v4a, **kw) == status


def test_evict_entry_numbers_that_do_not_fit(v4a):
    last = (1 << 31) - 32
    assert evict(v4a, first_entry=last + 1) == INVALID and b"first_entry" in v4a.lib.v4a_last_error()
    assert evict(v4a, first_entry=last, kept=None) == INVALID and b"first_entry" not in v4a.lib.v4a_last_error()  # 32 rows: they fit
    for kw in (dict(own_entry=8 * FAKE), dict(entry_out=None)):  # not used
        assert evict(v4a, first_entry=last + 1, kept=None, **kw) == INVALID and b"first_entry" not in v4a.lib.v4a_last_error()


def test_null_structs(v4a):
    L = v4a.lib
    s = shape(v4a)
    assert L.v4a_hca_attend_shared(FAKE, None, FAKE, 0, None, 1, FAKE, 1 << 40, None, None, ctypes.byref(s), None) == INVALID
    assert L.v4a_attend_weights(FAKE, None, FAKE, FAKE, FAKE, 1.0, 1, None, ctypes.byref(s), None) == INVALID
    assert L.v4a_evict(None, 1, 1, 0, 0, None, None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes(v4a):
    import torch
    x = torch.zeros((1, 2, 4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        v4a.v4a_rope([(x, x)], rope_dims=64)
    with pytest.raises(ValueError, match="one shape"):
        v4a.v4a_rope([(x, x[:, :1])], rope_dims=64)
    with pytest.raises(ValueError, match="n_q"):
        v4a.v4a_hca_attend_shared(x[0], None, None, None, x, m=128, window=0, ctx_len=1024)
    with pytest.raises(ValueError, match="rows"):
        v4a.v4a_evict(x[0, 0], x, x, x, x, x, budget=1)
