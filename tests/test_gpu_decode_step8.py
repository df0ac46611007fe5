"""The decode step with norms, a cache of 8 bits and drawn tokens: each call's output against
its definition in 64 bits on the inputs that the calls before it made, over several steps.
Tolerances as in the operators' own tests."""
import math

import pytest
import torch

import cache8_ref
import test_gpu_sample

pytestmark = pytest.mark.gpu

SIZES = dict(hidden=256, Hq=8, Hkv=2, D=64, vocab=1003, adapters=3, rank=8, page=16)


def step8(batch=5, prefix=144, max_own=40, seed=3, **kw):
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    return DecodeStep(batch, prefix, max_own, seed=seed, **{**SIZES, "norms": True, "cache": "e4m3", **kw})


def inputs(n, batch, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn((batch, 256), generator=g, device="cuda").half(), torch.rand((batch,), generator=g, device="cuda"))
            for _ in range(n)]


@pytest.mark.parametrize("D", [64, 128])
def test_steps_against_definitions(D):
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    net = step8(D=D)
    Hq, Hkv, prefix = 8, 2, 144
    for step, (x, u) in enumerate(inputs(36, 5)):     # across two borders of blocks and pages
        before = {n: getattr(net, n).clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
        at = net.own_len.clone()
        slots = net.own_table.gather(1, (at // 16).long()[:, None])[:, 0].long() * 16 + at % 16
        r = net.step(x, u=u)
        qr, kr, vr = cache8_ref.heads(r["qkv"], (at + prefix)[None], net.table, [0] * (D // 2), Hkv, D, False, net.q_norm, net.k_norm, 1e-6)
        off = 2.0 ** -19 * 1.5 * max(float(qr.abs().max()), float(kr.abs().max()))
        assert bool(((r["q"].double() - qr).abs() <= 2.0 ** -11 * qr.abs() + off + 2.0 ** -25).all())
        for name, new, err in (("k", kr, off), ("v", vr, 0.0)):
            codes, scale, wanted = cache8_ref.append(new, slots, before[name + "_cache"], before[name + "_scale"])
            have = getattr(net, name + "_cache").double().reshape(codes.shape)
            assert torch.equal(getattr(net, name + "_scale").double().reshape(scale.shape), scale), (step, name)
            old = ~torch.isnan(codes)
            assert torch.equal(have[old], codes[old]), (step, name)
            s = scale.repeat_interleave(16, 0)[:, :, None].expand_as(codes)
            half = (wanted.abs() * 2.0 ** -4).maximum(s * 2.0 ** -10) + err
            assert bool(((have * s - wanted).abs() <= half)[~old].all()), (step, name)
        lens = net.own_len + prefix
        o, bound, floor = cache8_ref.attention(r["q"].view(5, 1, Hq, D), net.k_cache, net.v_cache, net.k_scale, net.v_scale,
                                               net.page_table, lens, D ** -0.5)
        got = r["o"].view(5, 1, Hq, D).double()
        tol = 2.0 ** -11 * o.abs() + (2.0 ** -11 + 2.0 ** -13) * bound + 2.0 ** -25 * floor + 2.0 ** -24
        assert bool(((got - o).abs() <= tol).all()), step
        token = test_gpu_sample.check(dict(logits=r["logits"], u=u, temperature=net.temperature, top_k=net.top_k, top_p=net.top_p,
                                           min_p=net.min_p))
        assert torch.equal(token, r["token"]) and bool(torch.isfinite(r["logits"].gather(1, token.long()[:, None])).all())
        assert torch.equal(net.tokens.gather(1, at.long()[:, None])[:, 0], r["token"])
    assert q.error_flags(clear=True) == 0


def test_norms_with_a_cache_of_16_bits():
    net = step8(prefix=130, cache="f16")
    for x, u in inputs(3, 5):
        at = net.own_len.clone()
        r = net.step(x, u=u)
        qr, kr, vr = cache8_ref.heads(r["qkv"], (at + 130)[None], net.table, [0] * 32, 2, 64, False, net.q_norm, net.k_norm, 1e-6)
        off = 2.0 ** -19 * 1.5 * float(qr.abs().max().maximum(kr.abs().max()))
        assert bool(((r["q"].double() - qr).abs() <= 2.0 ** -11 * qr.abs() + off + 2.0 ** -25).all())
        slots = net.own_table.gather(1, (at // 16).long()[:, None])[:, 0].long() * 16 + at % 16
        assert bool(((net.k_cache.view(-1, 2, 64)[slots].double() - kr).abs() <= 2.0 ** -11 * kr.abs() + off + 2.0 ** -25).all())
        assert torch.equal(net.v_cache.view(-1, 2, 64)[slots], vr.half())


def test_the_two_caches_nearly_agree():
    """The same step with either cache: codes are within 2^-4 of the values, so outputs are near each other (a check
    that both read what the other writes, not of rounding)."""
    a, b = step8(), step8(cache="f16")
    x, u = inputs(1, 5)[0]
    oa, ob = a.step(x)["o"].float(), b.step(x)["o"].float()
    assert float((oa - ob).norm() / ob.norm()) < 2.0 ** -3


def test_whole_step_in_a_cuda_graph_gives_the_same():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    plain, net = step8(6, seed=12), step8(6, seed=12)
    x, u = inputs(1, 6)[0]
    expected = [plain.step(x, u=u) for _ in range(20)]
    first = net.step(x, u=u)
    assert all(torch.equal(expected[0][n], first[n]) for n in first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = net.step(x, u=u)
    for step in range(1, 20):
        graph.replay()
        for name in captured:
            assert torch.equal(captured[name], expected[step][name]), (step, name)
    assert torch.equal(net.k_cache.view(torch.uint8), plain.k_cache.view(torch.uint8)) and torch.equal(net.k_scale, plain.k_scale)
    assert q.error_flags(clear=True) == 0


def test_steps_with_overlapping_launches_give_the_same():
    """Programmatic overlap between the calls of a step: every launch waits for what it reads."""
    import gemm_qmv_quantize_gb300 as q
    results = []
    for overlap in (False, True):
        net = step8(6, 704, 32, seed=9)
        xs = inputs(20, 6, 2)
        torch.cuda.synchronize()
        try:
            q.set_launch_overlap(overlap)
            out = [net.step(x, u=u) for x, u in xs]
            torch.cuda.synchronize()
        finally:
            q.set_launch_overlap(False)
        results.append(out)
    for a, b in zip(*results):
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_more_replays_than_there_is_room_for_are_flagged():
    import gemm_qmv_quantize_gb300 as q
    net = step8(3, 48, 5, seed=13)
    x, u = inputs(1, 3)[0]
    net.step(x, u=u)
    torch.cuda.synchronize()
    q.error_flags(clear=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        net.step(x, u=u)
    for _ in range(4):
        graph.replay()
    assert q.error_flags(clear=True) == 0
    graph.replay()
    assert q.error_flags(clear=True) == 2


def test_two_captured_graphs_that_share_a_workspace():
    """One after the other: nothing in the workspace is expected from a call before."""
    import gemm_qmv_quantize_gb300 as q
    from test_gpu_paged_attention_e4m3 import inputs as attention
    cases = [attention(4, 1, 8, 2, 128, [900, 33, 0, 411], 32, seed=1), attention(2, 3, 20, 4, 64, [2000, 77], 16, seed=2)]
    ws = torch.empty((max(q.qmv_paged_attention_e4m3_workspace(*a["q"].shape[:3], a["k_cache"].shape[2], a["q"].shape[3], 4096)
                          for a in cases),), dtype=torch.uint8, device="cuda")
    plain = [q.qmv_paged_attention_e4m3(**a) for a in cases]
    graphs = []
    for a in cases:
        graphs.append((torch.cuda.CUDAGraph(), torch.empty_like(a["q"])))
        with torch.cuda.graph(graphs[-1][0]):
            q.qmv_paged_attention_e4m3(**a, out=graphs[-1][1], workspace=ws)
    for _ in range(3):
        for (graph, out), p in zip(graphs, plain):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, p)


def call_without_buffers(which):
    """A call without an output or a workspace: (call, bytes of its output, of its workspace)."""
    import gemm_qmv_quantize_gb300 as q
    from test_gpu_paged_attention_e4m3 import inputs as attention
    g = torch.Generator(device="cuda").manual_seed(8)
    if which == "attention":
        a = attention(8, 300, 32, 4, 128, [900] * 8, 32, seed=3)
        return (lambda s: q.qmv_paged_attention_e4m3(**a, stream=s), 8 * 300 * 32 * 128 * 2,
                q.qmv_paged_attention_e4m3_workspace(8, 300, 32, 4, 128, a["table"].shape[1] * 32))
    if which == "sample":
        x, u = torch.randn((20000, 500), generator=g, device="cuda"), torch.rand((20000,), generator=g, device="cuda")
        return lambda s: q.qmv_sample(x, u, stream=s), 20000 * 4, None
    table, slots = q.qmv_rope_table(64, 128, device="cuda"), torch.arange(2048, device="cuda")
    qkv, positions = torch.randn((2048, 24 * 128), generator=g, device="cuda"), torch.zeros((1, 2048), dtype=torch.int32, device="cuda")
    k, ks = cache8_ref.random_cache(g, 130, 16, 4, 128)
    k16, w = torch.zeros((130, 16, 4, 128), device="cuda").half(), torch.ones((128,), device="cuda")
    if which == "append":
        return (lambda s: q.qmv_rope_append_e4m3(qkv, positions, table, bytes(64), slots, k, k.clone(), ks, ks.clone(), stream=s),
                2048 * 16 * 128 * 2, None)
    return (lambda s: q.qmv_norm_rope_append(qkv, positions, table, bytes(64), slots, k16, k16, w, w, stream=s), 2048 * 16 * 128 * 2, None)


@pytest.mark.parametrize("handle", [lambda s: s, lambda s: s.cuda_stream], ids=["stream", "handle"])
@pytest.mark.parametrize("which", ["attention", "sample", "append", "norm"])
def test_buffers_of_a_call_are_its_streams_own(which, handle):
    """Blocks that the current stream has freed, which its queued work may still use, are
    neither written nor handed out by a call on another stream."""
    call, *sizes = call_without_buffers(which)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    plain = call(None)
    torch.cuda.synchronize()
    freed = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes if n]
    places = [t.data_ptr() for t in freed]
    torch.cuda.synchronize()
    del freed
    out = call(handle(s))
    s.synchronize()
    assert out.data_ptr() not in places
    again = [torch.empty((n,), dtype=torch.uint8, device="cuda") for n in sizes if n]
    assert [t.data_ptr() for t in again] == places
    for t in again:
        assert bool((t == 7).all())
    assert torch.equal(out, plain)
