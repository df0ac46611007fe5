"""GPU tests of qmv_rope_append against its definition in 64 bits.

Tolerance: a c - b s in fp32 is within 2^-22 (|a c| + |b s|) of its value; then one
rounding to the 16-bit type (2^-11 for binary16, 2^-8 for bfloat16, 2^-25 below
binary16's normal range). Copied elements are rounded once: equal to the conversion.
"""
import pytest
import torch

import decode_ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": (torch.float16, 2.0 ** -11), "bf16": (torch.bfloat16, 2.0 ** -8)}


def inputs(M, Hq, Hkv, D, rot, axes=1, type_="f16", seed=0, n_positions=300, page=16):
    import gemm_qmv_quantize_gb300 as q
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[type_][0]
    pages = (M + 30) // page + 1
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:M]
    if M > 2:
        slots[1] = -1
    return dict(qkv=r(M, (Hq + 2 * Hkv) * D),
                positions=torch.randint(0, n_positions, (axes, M), generator=g, device="cuda", dtype=torch.int32),
                table=q.qmv_rope_table(n_positions, rot, 10000.0, "cuda"),
                axis_of_pair=[i % axes for i in range(rot // 2)], slots=slots,
                k_cache=r(pages, page, Hkv, D).to(dtype), v_cache=r(pages, page, Hkv, D).to(dtype))


def check(args, type_, interleaved):
    import gemm_qmv_quantize_gb300 as q
    Hkv, D = args["k_cache"].shape[2:]
    k0, v0 = args["k_cache"].clone(), args["v_cache"].clone()
    got = q.qmv_rope_append(**args, interleaved=interleaved)
    qr, kr, vr = decode_ref.rope(args["qkv"], args["positions"], args["table"], args["axis_of_pair"], Hkv, D, interleaved)
    big = float(args["qkv"].abs().max())
    u = TYPES[type_][1]
    close = lambda x, y: bool(((x.double() - y).abs() <= u * y.abs() + 2.0 ** -21 * big + 2.0 ** -25).all())  # noqa: E731
    assert close(got, qr)
    live = args["slots"] >= 0
    to = args["slots"][live]
    k, v = (c.view(-1, Hkv, D) for c in (args["k_cache"], args["v_cache"]))
    assert close(k[to], kr[live])
    assert torch.equal(v[to], vr[live].to(v.dtype))
    others = torch.ones((k.shape[0],), dtype=torch.bool, device="cuda")
    others[to] = False
    assert torch.equal(k[others], k0.view(-1, Hkv, D)[others]) and torch.equal(v[others], v0.view(-1, Hkv, D)[others])


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,Hq,Hkv,D,rot,axes", [
    (1, 32, 32, 128, 128, 1), (1, 1, 1, 8, 8, 1), (3, 5, 1, 64, 64, 2), (17, 40, 8, 128, 128, 3), (9, 6, 2, 80, 40, 3),
    (4, 3, 3, 256, 256, 4), (5, 8, 2, 96, 0, 1), (130, 7, 1, 64, 32, 1), (2, 28, 4, 128, 8, 3)])
def test_sizes_types_and_orders(M, Hq, Hkv, D, rot, axes, type_, interleaved):
    check(inputs(M, Hq, Hkv, D, rot, axes, type_, seed=M + D), type_, interleaved)


def test_position_zero_is_the_conversion():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(4, 4, 2, 64, 64)
    args["positions"].zero_()
    got = q.qmv_rope_append(**args)
    assert torch.equal(got, args["qkv"].view(4, 8, 64)[:, :4].half())


def test_empty_and_all_padding():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(0, 4, 2, 64, 64)
    assert q.qmv_rope_append(**args).shape == (0, 4, 64)
    args = inputs(5, 4, 2, 64, 64)
    args["slots"].fill_(-3)
    check(args, "f16", False)


def test_indices_outside_are_flagged_and_not_followed():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    args = inputs(3, 4, 2, 64, 64, seed=4)
    args["positions"][0] = torch.tensor([10 ** 9, 5, -1], dtype=torch.int32)
    args["slots"][:] = torch.tensor([0, 1 << 40, 2])
    k0 = args["k_cache"].clone()
    got = q.qmv_rope_append(**args)
    assert q.error_flags(clear=True) == 2
    ends = {**args, "positions": torch.tensor([[299, 5, 0]], dtype=torch.int32, device="cuda"),
            "slots": torch.tensor([0, -1, 2], device="cuda"), "k_cache": k0, "v_cache": args["v_cache"].clone()}
    assert torch.equal(got, q.qmv_rope_append(**ends))
    assert torch.equal(args["k_cache"], ends["k_cache"])
    assert q.error_flags(clear=True) == 0


def test_refusals():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(2, 4, 2, 64, 64, axes=2)
    with pytest.raises(ValueError):
        q.qmv_rope_append(**{**args, "qkv": args["qkv"][:, :250].contiguous()})   # not whole heads
    with pytest.raises(ValueError):
        q.qmv_rope_append(**{**args, "axis_of_pair": [0] * 31})
    with pytest.raises(TypeError):
        q.qmv_rope_append(**{**args, "positions": args["positions"].long()})
    with pytest.raises(TypeError):
        q.qmv_rope_append(**{**args, "v_cache": args["v_cache"].bfloat16()})
    with pytest.raises(q.QmvError):
        q.qmv_rope_append(**{**args, "axis_of_pair": [2] * 32})                   # axis without positions
    with pytest.raises(q.QmvError):
        q.qmv_rope_append(**inputs(2, 4, 2, 60, 24))                              # D not a multiple of 8
    with pytest.raises(q.QmvError):
        q.qmv_rope_append(**inputs(2, 4, 2, 64, 20))                              # rot not a multiple of 8
