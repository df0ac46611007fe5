"""The decode step's operators together, as gemm_qmv_quantize_gb300/decode_step.py runs
them: each call's output against its definition in 64 bits on the inputs that the calls
before it made, over several steps. Tolerances as in the operators' own tests."""
import math

import pytest
import torch

import decode_ref
import oracle

pytestmark = pytest.mark.gpu


def test_steps_against_definitions():
    import gemm_qmv_quantize_gb300 as q
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    q.error_flags(clear=True)
    hidden, Hq, Hkv, D, V, B, prefix = 256, 8, 2, 64, 1003, 5, 130
    net = DecodeStep(B, prefix, 24, hidden=hidden, Hq=Hq, Hkv=Hkv, D=D, vocab=V, adapters=3, rank=8, page=16, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    for step in range(20):
        x = torch.randn((B, hidden), generator=g, device="cuda").half()
        tokens, total = net.tokens.clone(), net.own_len.clone()
        r = net.step(x)

        def projected(name, inp, got):
            codes, scales, gs = net.w[name]
            y, bound = oracle.nvfp4_w4a16(codes.cpu().numpy(), scales.cpu().numpy(), gs, inp.cpu().numpy())
            y, bound = torch.from_numpy(y).cuda(), torch.from_numpy(bound).cuda()
            if name in net.a:
                y, more = decode_ref.lora(inp, net.a[name], net.b[name], net.adapter, net.scale, y)
                bound = bound + more
            assert bool(((got.double() - y).abs() <= 1e-3 * bound + 1e-6).all()), (step, name)

        projected("qkv", x, r["qkv"])
        position = (net.own_len - 1 + prefix)[None]
        qr, kr, vr = decode_ref.rope(r["qkv"], position, net.table, [0] * (D // 2), Hkv, D, False)
        u = 2.0 ** -11
        near = lambda a, b: bool(((a.double() - b).abs() <= u * b.abs() + 2.0 ** -20 * float(r["qkv"].abs().max()) + 2.0 ** -25).all())  # noqa: E731
        assert near(r["q"], qr)
        for b in range(B):
            page, at = int(net.own_table[b, (int(net.own_len[b]) - 1) // 16]), (int(net.own_len[b]) - 1) % 16
            assert near(net.k_cache[page, at], kr[b]) and near(net.v_cache[page, at], vr[b])
        o, bound = decode_ref.attention(r["q"].view(B, 1, Hq, D), net.k_cache, net.v_cache, net.prefix_table, prefix,
                                        net.own_table, net.own_len, 1 / math.sqrt(D))
        got = r["o"].view(B, 1, Hq, D).double()
        assert bool(((got - o).abs() <= u * o.abs() + (u + 2e-3) * bound + 2.0 ** -24).all()), step
        projected("o", r["o"], r["hidden"])
        projected("head", r["hidden"].half(), r["raw"])
        y = decode_ref.logits(r["raw"], tokens, net.prompt_len, total, net.repetition, net.presence, net.frequency, None,
                              None, net.mask, net.mask_row)
        logits = r["logits"].double().cpu()
        fine = torch.isfinite(y)
        assert torch.equal(logits[~fine], y[~fine])
        big = 2 * r["raw"].double().abs().cpu() + 30.0
        assert bool(((logits - y).abs()[fine] <= 2.0 ** -22 * big[fine]).all())
        assert torch.equal(net.tokens.gather(1, total.long()[:, None])[:, 0].long().cpu(), logits.argmax(1))
    assert int(net.own_len[0]) == 20
    assert q.error_flags(clear=True) == 0


def test_step_in_a_cuda_graph_gives_the_same():
    """A step's calls, captured once and replayed."""
    import gemm_qmv_quantize_gb300 as q
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    net = DecodeStep(4, 200, 32, hidden=256, Hq=8, Hkv=2, D=64, vocab=1003, adapters=3, rank=8, page=16, seed=5)
    x = torch.randn((4, 256), device="cuda").half()
    q_ = torch.randn((4, 1, 8, 64), device="cuda").half()
    own = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    run = lambda: (net.project("qkv", x), q.qmv_prefix_attention(  # noqa: E731
        q_, net.k_cache, net.v_cache, net.prefix_table, 200, net.own_table, own, max_own=32, workspace=net.workspace))
    plain = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(plain, captured):
        assert torch.equal(a, b)


def test_steps_with_overlapping_launches_give_the_same():
    """Programmatic overlap between the calls of a step: every launch waits for what it reads."""
    import gemm_qmv_quantize_gb300 as q
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    results = []
    for overlap in (False, True):
        net = DecodeStep(6, 700, 32, hidden=512, Hq=8, Hkv=2, D=64, vocab=4001, adapters=3, rank=16, page=16, seed=9)
        g = torch.Generator(device="cuda").manual_seed(2)
        xs = [torch.randn((6, 512), generator=g, device="cuda").half() for _ in range(12)]
        torch.cuda.synchronize()
        try:
            q.set_launch_overlap(overlap)
            out = [net.step(x) for x in xs]
            torch.cuda.synchronize()
        finally:
            q.set_launch_overlap(False)
        results.append(out)
    for a, b in zip(*results):
        for name in a:
            assert torch.equal(a[name], b[name]), name


def calls_without_buffers():
    """Each operator without an output or a workspace: (call, bytes of its output, of its workspace)."""
    import gemm_qmv_quantize_gb300 as q
    rand = lambda *s, dtype=torch.float32: torch.randn(s, device="cuda").to(dtype)  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    half, M, N, K = torch.float16, 64, 1 << 16, 512
    x, a, b, base = rand(M, K, dtype=half), rand(2, 32, K, dtype=half), rand(2, N, 32, dtype=half), rand(M, N)
    scale, adapter = rand(2), torch.arange(M, dtype=torch.int32, device="cuda") % 2
    qkv, table = rand(2048, 24 * 128), q.qmv_rope_table(64, 128, device="cuda")
    k, v = rand(200, 16, 4, 128, dtype=half), rand(200, 16, 4, 128, dtype=half)
    slots, positions = torch.arange(2048, device="cuda"), torch.zeros((1, 2048), dtype=torch.int32, device="cuda")
    qa, pages = rand(2, 200, 32, 128, dtype=half), torch.arange(200, dtype=torch.int32, device="cuda")
    own_table, own_len = pages[:26].reshape(2, 13).contiguous(), ints(200, 208)
    x2, tokens, one = rand(40, 100000), ints(*[1] * 40).reshape(40, 1), ints(*[1] * 40)
    return [
        (lambda s: q.qmv_lora_add(x, a, b, adapter, scale, base, stream=s), M * N * 4, q.qmv_lora_add_workspace(M, 32, K)),
        (lambda s: q.qmv_rope_append(qkv, positions, table, bytes(64), slots, k, v, stream=s), 2048 * 16 * 128 * 2, None),
        (lambda s: q.qmv_prefix_attention(qa, k, v, pages, 3000, own_table, own_len, stream=s), 2 * 200 * 32 * 128 * 2,
         q.qmv_prefix_attention_workspace(2, 200, 32, 4, 128, 3000, 208)),
        (lambda s: q.qmv_penalize_logits(x2, tokens, one, one, stream=s), 40 * 100000 * 4, None)]


def raw(s):
    return s.cuda_stream


@pytest.mark.parametrize("handle", [lambda s: s, raw], ids=["stream", "handle"])
@pytest.mark.parametrize("which", range(4))
def test_buffers_of_a_call_are_its_streams_own(which, handle):
    """Blocks that the current stream has freed, which its queued work may still use, are
    neither written nor handed out by a call on another stream."""
    call, *sizes = calls_without_buffers()[which]
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


def test_more_replays_than_there_is_room_for_are_flagged():
    """The last token's place is taken again: nothing is written or read out of range."""
    import gemm_qmv_quantize_gb300 as q
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    net = DecodeStep(3, 40, 5, hidden=256, Hq=8, Hkv=2, D=64, vocab=1003, adapters=3, rank=8, page=16, seed=13)
    x = torch.randn((3, 256), device="cuda").half()
    net.step(x)
    torch.cuda.synchronize()
    q.error_flags(clear=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        net.step(x)
    for _ in range(4):
        graph.replay()
    assert q.error_flags(clear=True) == 0
    graph.replay()
    assert q.error_flags(clear=True) == 2


def test_whole_step_in_a_cuda_graph_gives_the_same():
    """step(), captured once and replayed: every operator and the projections between them."""
    import gemm_qmv_quantize_gb300 as q
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    q.error_flags(clear=True)
    plain, net = (DecodeStep(6, 300, 16, hidden=256, Hq=8, Hkv=2, D=64, vocab=1003, adapters=3, rank=8, page=16, seed=12)
                  for _ in range(2))
    x = torch.randn((6, 256), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").half()
    expected = [plain.step(x) for _ in range(8)]
    first = net.step(x)
    assert all(torch.equal(expected[0][n], first[n]) for n in first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = net.step(x)
    for step in range(1, 8):
        graph.replay()
        for name in captured:
            assert torch.equal(captured[name], expected[step][name]), (step, name)
    assert torch.equal(net.tokens, plain.tokens) and torch.equal(net.own_len, plain.own_len)
    assert q.error_flags(clear=True) == 0
