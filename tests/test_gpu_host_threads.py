"""Calls whose host thread has not used CUDA before."""
import threading

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
    """name -> (call, its output).  Nothing but the call touches CUDA: every tensor is there, the workspaces too."""
    g = torch.Generator().manual_seed(4)
    normal = lambda *s: torch.randn(s, generator=g).to(BF16).cuda()
    B, N, d, H = 1, 300, 512, 64
    q, ent, tok = normal(B, 1, H, d), normal(B, N, d), normal(B, 128, d)
    qi, w, ki = normal(B, 1, 16, 128), torch.rand((B, 1, 16), generator=g).cuda(), normal(B, N, 128)
    codes, exps = torch.zeros((B, N, 64), dtype=torch.uint8, device="cuda"), torch.zeros((B, N, 4), dtype=torch.uint8, device="cuda")
    v4a.v4a_quantize_mxfp4(ki, codes, exps)
    sel = torch.arange(0, 128, dtype=torch.int32).repeat(B, 1, 1).cuda()
    lse = torch.full((B, 1, H), 4.0, device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    scores, scores4 = (torch.zeros((B, 1, N), device="cuda") for _ in range(2))
    idx, idx4 = (torch.zeros((B, 1, 32), dtype=torch.int32, device="cuda") for _ in range(2))
    csa, hca = (torch.zeros((B, 1, H, d), device="cuda") for _ in range(2))
    shared, weights, x = torch.zeros_like(q), torch.zeros((B, N), device="cuda"), normal(B, 1, 4, 64)
    turned = torch.zeros_like(x)
    return {
        "index_scores": (lambda: v4a.v4a_index_scores(qi, w, ki, None, scores, m=4, ctx_len=4 * N), scores),
        "index_scores_mxfp4": (lambda: v4a.v4a_index_scores_mxfp4(qi, w, codes, exps, scores4, m=4, ctx_len=4 * N), scores4),
        "topk": (lambda: v4a.v4a_topk(qi, w, ki, None, idx, m=4, k=32, ctx_len=4 * N, workspace=ws), idx),
        "topk_mxfp4": (lambda: v4a.v4a_topk_mxfp4(qi, w, codes, exps, idx4, m=4, k=32, ctx_len=4 * N, workspace=ws), idx4),
        "csa_attend": (lambda: v4a.v4a_csa_attend(q, ent, sel, tok, 4 * N - 128, csa, m=4, window=128, ctx_len=4 * N, workspace=ws), csa),
        "hca_attend": (lambda: v4a.v4a_hca_attend(q, ent, tok, 128 * N - 128, hca, m=128, window=128, ctx_len=128 * N, workspace=ws), hca),
        "hca_attend_shared": (lambda: v4a.v4a_hca_attend_shared(q, ent[0], None, None, shared, m=128, window=0, ctx_len=128 * N, workspace=ws), shared),
        "attend_weights": (lambda: v4a.v4a_attend_weights(q, ent, lse, None, weights, m=128, ctx_len=128 * N, decay=0.0), weights),
        "rope": (lambda: v4a.v4a_rope([(x, turned)], rope_dims=64, pos0=5), turned),
    }


@pytest.mark.parametrize("name", ["index_scores", "index_scores_mxfp4", "topk", "topk_mxfp4", "csa_attend", "hca_attend", "hca_attend_shared",
                                  "attend_weights", "rope"])
def test_first_call_of_a_host_thread(v4a, name):
    call, out = calls(v4a)[name]
    call()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    said = []

    def run():
        try:
            call()
        except Exception as e:
            said.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not said
    assert torch.equal(out, want) and want.any()
