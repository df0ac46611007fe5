"""Calls of one operator on two streams at once, each with buffers of its own, give what they give one after another."""
import pytest
import torch

import cache8_ref
import test_gpu_append_e4m3
import test_gpu_paged_attention_e4m3
import test_gpu_sample

pytestmark = pytest.mark.gpu


def attention(lens, T, seed):
    import gemm_qmv_quantize_gb300 as q
    a = test_gpu_paged_attention_e4m3.inputs(len(lens), T, 16, 4, 128, lens, 64, "f16", seed=seed)
    out, n = torch.empty_like(a["q"]), a["table"].shape[1] * 64
    ws = torch.empty((q.qmv_paged_attention_e4m3_workspace(len(lens), T, 16, 4, 128, n),), dtype=torch.uint8, device="cuda")
    return lambda s: [q.qmv_paged_attention_e4m3(**a, out=out, workspace=ws, stream=s)]


def sample(M, V, seed, **filters):
    import gemm_qmv_quantize_gb300 as q
    a = test_gpu_sample.inputs(M, V, 3.0, seed=seed, **filters)
    out, prob = torch.empty((M,), dtype=torch.int32, device="cuda"), torch.empty((M,), device="cuda")
    return lambda s: [q.qmv_sample(**a, out=out, prob=prob, stream=s), prob]


def append(M, seed):
    import gemm_qmv_quantize_gb300 as q
    a = test_gpu_append_e4m3.inputs(list(range(3, 3 + M)), Hq=8, D=128, page=64, pages=M // 64 + 2, seed=seed)
    out = torch.empty((M, 8, 128), dtype=torch.float16, device="cuda")

    def call(s):     # (again and again the same: q, codes and scales)
        q.qmv_rope_append_e4m3(**a, out=out, stream=s)
        return [out] + [a[n].view(torch.uint8) for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    return call


@pytest.mark.parametrize("make", [
    lambda: (attention([9000, 17, 4000], 1, 1), attention([3000, 2222], 3, 2)),          # runs over all SMs
    lambda: (attention([500], 1, 3), attention([300, 700], 1, 4)),                       # clusters
    lambda: (attention([20000] * 4, 1, 5), sample(40, 151936, 6, top_p=0.9)),
    lambda: (sample(30, 50257, 7, top_k=50), sample(17, 151936, 8, top_k=1000, top_p=0.95)),
    lambda: (append(1000, 9), append(700, 10)), lambda: (append(2000, 11), attention([6000, 6000], 1, 12))],
    ids=["runs", "clusters", "attention and sampling", "sampling", "appends", "append and attention"])
def test_two_calls_at_once(make):
    calls = make()
    plain = [[t.clone() for t in call(None)] for call in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        results = [call(s) for call, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for p, r in zip(plain, results):
        for a, b in zip(p, r):
            assert torch.equal(a, b)
