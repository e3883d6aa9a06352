"""Calls on a stream that is not the current one, without a workspace of the caller's."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def v4a():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import compressed_sparse_long_v4a_b200 as v
    return v


def calls(v4a):
    """name -> (call(out, stream), its output, bytes of workspace)"""
    g = torch.Generator().manual_seed(3)
    normal = lambda *s: torch.randn(s, generator=g).to(BF16).cuda()
    B, N, d, H = 2, 1200, 512, 64
    q, ent, tok = normal(B, 1, H, d), normal(B, N, d), normal(B, 128, d)
    qi, w, ki = normal(B, 1, 16, 128), torch.rand((B, 1, 16), generator=g).cuda(), normal(B, N, 128)
    sel = torch.arange(0, 512, 4, dtype=torch.int32).repeat(B, 1, 1).cuda()
    L = 4 * N
    return {
        "topk": (lambda o, s: v4a.v4a_topk(qi, w, ki, None, o, m=4, k=128, ctx_len=L, stream=s),
                 torch.zeros((B, 1, 128), dtype=torch.int32, device="cuda"), v4a.v4a_workspace_size("topk", batch=B, m=4, k=128, ctx_len=L, heads_i=16, d_i=128)),
        "csa": (lambda o, s: v4a.v4a_csa_attend(q, ent, sel, tok, L - 128, o, m=4, window=128, ctx_len=L, stream=s),
                torch.zeros((B, 1, H, d), device="cuda"), v4a.v4a_workspace_size("csa_attend", batch=B, heads=H, d=d, m=4, k=128, window=128, ctx_len=L)),
        "hca": (lambda o, s: v4a.v4a_hca_attend(q, ent, tok, 128 * N - 128, o, m=128, window=128, ctx_len=128 * N, stream=s),
                torch.zeros((B, 1, H, d), device="cuda"), v4a.v4a_workspace_size("hca_attend", batch=B, heads=H, d=d, m=128, window=128, ctx_len=128 * N)),
    }


@pytest.mark.parametrize("name", ["topk", "csa", "hca"])
@pytest.mark.parametrize("raw", [False, True])
def test_workspace_takes_no_memory_that_the_current_stream_still_uses(v4a, name, raw):
    # a temporary of the current stream, let go of while kernels that read it are queued: its block may serve that stream
    # again at once, but no other
    call, out, size = calls(v4a)[name]
    call(out, None)
    want = out.clone()
    copy = torch.empty(size, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        tmp = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(20_000_000)  # 10 ms: the call below is done long before
        copy.copy_(tmp)
        del tmp
        call(out, side.cuda_stream if raw else side)
        side.synchronize()
        assert torch.equal(out, want)
        assert (copy == 7).all()


def test_default_stream_while_another_is_current(v4a):
    call, out, _ = calls(v4a)["hca"]
    call(out, None)
    want = out.clone()
    torch.cuda.synchronize()
    for stream in (0, 1, torch.cuda.default_stream()):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            call(out, stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_capture_on_another_stream_needs_a_workspace(v4a):
    call, out, _ = calls(v4a)["hca"]
    call(out, None)
    torch.cuda.synchronize()
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out.add_(1.0)
        with torch.cuda.stream(other):
            with pytest.raises(ValueError, match="workspace"):
                call(out, side)
        call(out, side)  # the current stream: the graph's own pool
    graph.replay()
    torch.cuda.synchronize()
