"""Two host threads calling the C ABI at once, each on a stream of its own, with sizes that ask for different amounts of
shared memory of the same kernel: every call succeeds and gives what it gives alone."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
CALLS = 4000


@pytest.fixture(scope="module")
def v4a():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import compressed_sparse_long_v4a_b200 as v
    return v


def together(jobs, calls=CALLS):
    """jobs: (call(stream) -> status, its outputs).  Runs each alone, then all of them at once, over and over."""
    streams = [torch.cuda.Stream() for _ in jobs]
    alone = []
    for (call, outs), s in zip(jobs, streams):
        assert call(s.cuda_stream) == 0
        torch.cuda.synchronize()
        alone.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    failed, start = [0] * len(jobs), threading.Barrier(len(jobs))

    def run(i):
        start.wait()
        for _ in range(calls):
            failed[i] += jobs[i][0](streams[i].cuda_stream) != 0

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(jobs)
    for (_, outs), want in zip(jobs, alone):
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def evict_job(v4a, rows):
    g = torch.Generator().manual_seed(rows)
    own, w = torch.randn((1, rows, 8), generator=g).cuda(), torch.randn((1, rows), generator=g).cuda()
    budget = rows // 2
    outs = [torch.zeros((1, budget, 8), device="cuda"), torch.zeros((1, budget), device="cuda"),
            torch.zeros((1, budget), dtype=torch.int32, device="cuda"), torch.zeros((1,), dtype=torch.int32, device="cuda")]
    io = v4a.EvictIO(own.data_ptr(), w.data_ptr(), None, None, rows, 8, 0, outs[0].data_ptr(), outs[1].data_ptr(), None,
                     outs[2].data_ptr(), outs[3].data_ptr(), budget, 0)
    keep = (own, w, io)
    return (lambda s, keep=keep: v4a.lib.v4a_evict(ctypes.byref(keep[2]), 1, budget, 1, 1, None, s)), outs


def test_evict(v4a):
    together([evict_job(v4a, 8192), evict_job(v4a, 1000)])


def weights_job(v4a, heads):
    g = torch.Generator().manual_seed(heads)
    q, own = torch.randn((1, 1, heads, 512), generator=g).bfloat16().cuda(), torch.randn((1, 200, 512), generator=g).bfloat16().cuda()
    lse, out = torch.full((1, 1, heads), 4.0, device="cuda"), torch.zeros((1, 200), device="cuda")
    c = v4a.SharedCache(None, 0, own.data_ptr(), 200, None, None, None, 0, None)
    s = v4a.Shape(1, 1, heads, 512, 128, 0, 0, 128 * 200)
    keep = (q, own, lse, out, c, s)
    return (lambda st, keep=keep: v4a.lib.v4a_attend_weights(keep[0].data_ptr(), ctypes.byref(keep[4]), keep[2].data_ptr(), None,
                                                             keep[3].data_ptr(), 0.0, 1, None, ctypes.byref(keep[5]), st)), [out]


def test_weights(v4a):
    together([weights_job(v4a, 64), weights_job(v4a, 3), weights_job(v4a, 5)], 20000)


def scores_job(v4a, heads, d):
    g = torch.Generator().manual_seed(heads)
    q, w = torch.randn((1, 1, heads, d), generator=g).cuda(), torch.rand((1, 1, heads), generator=g).cuda()
    k, out = torch.randn((1, 64, d), generator=g).cuda(), torch.zeros((1, 1, 64), device="cuda")
    s = v4a.Shape(1, 1, 0, 0, 4, 0, 0, 256)
    keep = (q, w, k, out, s)
    return (lambda st, keep=keep: v4a.lib.v4a_index_scores(keep[0].data_ptr(), keep[1].data_ptr(), keep[2].data_ptr(), None,
                                                           keep[3].data_ptr(), heads, d, 0, 0, ctypes.byref(keep[4]), st)), [out]


def test_index_scores(v4a):
    together([scores_job(v4a, 64, 512), scores_job(v4a, 40, 8), scores_job(v4a, 36, 16)], 20000)
