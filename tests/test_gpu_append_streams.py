"""Appends with norms on a stream of their own: all that the call writes (q, codes or values, and scales) is
the current stream's call's, and the output comes from that stream's memory. Caches are made once, stand by
themselves and live until the stream is done."""
import pytest
import torch

import cache8_ref

pytestmark = pytest.mark.gpu

M, Hq, Hkv, D = 2048, 16, 4, 128


def caches(which):
    """(k, v, further arguments) of a call, filled."""
    g = torch.Generator(device="cuda").manual_seed(8)
    if which == "norm":
        return [torch.randn((130, 16, Hkv, D), generator=g, device="cuda").half() for _ in range(2)]
    (k, ks), (v, vs) = (cache8_ref.random_cache(g, 130, 16, Hkv, D) for _ in range(2))
    return [k, v, ks, vs]


def bits(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("handle", [lambda s: s, lambda s: s.cuda_stream], ids=["stream", "handle"])
@pytest.mark.parametrize("which", ["codes", "norm"])
def test_an_append_on_another_stream(which, handle):
    import gemm_qmv_quantize_gb300 as q
    fn = q.qmv_norm_rope_append if which == "norm" else q.qmv_rope_append_e4m3
    g = torch.Generator(device="cuda").manual_seed(9)
    qkv, w = torch.randn((M, (Hq + 2 * Hkv) * D), generator=g, device="cuda"), torch.rand((D,), generator=g, device="cuda") + 0.5
    positions = torch.randint(0, 64, (1, M), generator=g, device="cuda", dtype=torch.int32)
    table, slots = q.qmv_rope_table(64, D, device="cuda"), torch.arange(5, 5 + M, device="cuda")
    first, second = caches(which), caches(which)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(first, second))
    call = lambda cache, stream: fn(qkv, positions, table, bytes(D // 2), slots, *cache, w, w, stream=stream)  # noqa: E731
    s = torch.cuda.Stream()
    plain = call(first, None)
    torch.cuda.synchronize()
    freed = torch.full((plain.numel() * 2,), 7, dtype=torch.uint8, device="cuda")
    place = freed.data_ptr()
    torch.cuda.synchronize()
    del freed
    out = call(second, handle(s))
    s.synchronize()
    assert out.data_ptr() != place
    again = torch.empty((plain.numel() * 2,), dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == place and bool((again == 7).all())
    assert torch.equal(out, plain)
    for a, b in zip(first, second):
        assert torch.equal(bits(a), bits(b))
    assert not torch.equal(bits(first[0]), bits(caches(which)[0]))
