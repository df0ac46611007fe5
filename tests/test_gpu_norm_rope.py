"""GPU tests of qmv_norm_rope_append against its definition in 64 bits.

Tolerance: a head's sum of squares in fp32 is within 13 steps of 2^-24 of its value (8 in a
lane, 5 between lanes), the mean and eps add 2, the root halves that and with the quotient
adds 2, the two products 2: 12 in all; the turn adds 3 of |a c| + |b s| <= sqrt(2) times the largest
normed value: 2^-20 times twice that is above the sum. Then one rounding to 16 bits (2^-11 or
2^-8, 2^-25 below binary16's normal range). v is equal to the conversion.
"""
import pytest
import torch

import cache8_ref
from test_gpu_rope_append import TYPES, inputs

pytestmark = pytest.mark.gpu


def norms(D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    return dict(q_norm=torch.randn((D,), generator=g, device="cuda"), k_norm=torch.randn((D,), generator=g, device="cuda") + 1)


def check(args, type_="f16", eps=1e-6, interleaved=False, **kw):
    import gemm_qmv_quantize_gb300 as q
    Hkv, D = args["k_cache"].shape[2:]
    k0, v0 = args["k_cache"].clone(), args["v_cache"].clone()
    got = q.qmv_norm_rope_append(**args, eps=eps, interleaved=interleaved, **kw)
    qr, kr, vr = cache8_ref.heads(args["qkv"], args["positions"], args["table"], args["axis_of_pair"], Hkv, D, interleaved,
                                  args["q_norm"], args["k_norm"], eps)
    big = max([float(t.abs().max()) for t in (qr, kr) if t.numel()] + [0.0])
    u = TYPES[type_][1]
    close = lambda x, y: bool(((x.double() - y).abs() <= u * y.abs() + 2.0 ** -19 * 1.5 * big + 2.0 ** -25).all())  # noqa: E731
    assert close(got, qr)
    live = (args["slots"] >= 0) & (args["slots"] < k0.shape[0] * k0.shape[1])
    to = args["slots"][live]
    k, v = (c.view(-1, Hkv, D) for c in (args["k_cache"], args["v_cache"]))
    assert close(k[to], kr[live])
    assert torch.equal(v[to], vr[live].to(v.dtype))
    others = torch.ones((k.shape[0],), dtype=torch.bool, device="cuda")
    others[to] = False
    assert torch.equal(k[others], k0.view(-1, Hkv, D)[others]) and torch.equal(v[others], v0.view(-1, Hkv, D)[others])
    return got


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,Hq,Hkv,D,rot,axes", [
    (1, 32, 8, 128, 128, 1), (1, 1, 1, 8, 8, 1), (3, 5, 1, 64, 64, 2), (17, 40, 8, 128, 64, 3), (9, 6, 2, 80, 40, 3),
    (4, 3, 3, 256, 256, 4), (5, 8, 2, 96, 0, 1), (130, 7, 1, 24, 16, 1), (2, 28, 4, 136, 8, 3)])
def test_sizes_types_and_orders(M, Hq, Hkv, D, rot, axes, type_, interleaved):
    check({**inputs(M, Hq, Hkv, D, rot, axes, type_, seed=M + D), **norms(D, M)}, type_, interleaved=interleaved)


@pytest.mark.parametrize("type_,interleaved", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("M,Hq,Hkv,D,rot,axes", [
    (300, 4, 1, 128, 128, 1), (7400, 1, 1, 64, 64, 1), (3701, 5, 2, 80, 40, 3), (2501, 16, 4, 96, 0, 1), (3701, 2, 2, 256, 256, 4),
    (1100, 40, 8, 128, 64, 1), (9001, 3, 1, 8, 8, 1), (1001, 40, 8, 128, 128, 1)])
def test_long_prompts(M, Hq, Hkv, D, rot, axes, type_, interleaved):
    check({**inputs(M, Hq, Hkv, D, rot, axes, type_, seed=M + D), **norms(D, M)}, type_, interleaved=interleaved)
    check({**inputs(M, Hq, Hkv, D, rot, axes, type_, seed=M + D), **norms(D, M), "q_norm": None}, type_, interleaved=interleaved)


def test_indices_outside_in_a_long_prompt():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    args = {**inputs(8000, 4, 2, 64, 64, seed=5), **norms(64)}
    good = q.qmv_norm_rope_append(**args)
    assert q.error_flags(clear=True) == 0
    at = torch.tensor([0, 1, 1217, 7999], device="cuda")
    for bad in (10 ** 9, -1):
        positions = args["positions"].clone()
        positions[:, at] = bad
        got = q.qmv_norm_rope_append(**{**args, "positions": positions})
        assert q.error_flags(clear=True) == 2
        got[at] = good[at]
        assert torch.equal(got, good)
    k0 = args["k_cache"].clone()
    slots = torch.full_like(args["slots"], -1)
    slots[-1] = 1 << 40
    q.qmv_norm_rope_append(**{**args, "slots": slots})
    assert q.error_flags(clear=True) == 2 and torch.equal(args["k_cache"], k0)


@pytest.mark.parametrize("without", ["q_norm", "k_norm"])
def test_without_one_norm(without):
    check({**inputs(6, 8, 2, 128, 128), **norms(128), without: None})


def test_without_norms_the_same_as_rope_append():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(19, 12, 4, 64, 32, type_="bf16", seed=3)
    again = {**args, "k_cache": args["k_cache"].clone(), "v_cache": args["v_cache"].clone()}
    assert torch.equal(q.qmv_norm_rope_append(**args, q_norm=None, k_norm=None), q.qmv_rope_append(**again))
    assert torch.equal(args["k_cache"], again["k_cache"]) and torch.equal(args["v_cache"], again["v_cache"])


def test_zero_heads_and_a_large_eps():
    args = {**inputs(5, 4, 2, 64, 64), **norms(64)}
    args["qkv"][2] = 0
    got = check(args)
    assert bool((got[2] == 0).all())
    check({**inputs(5, 4, 2, 64, 64), **norms(64)}, eps=3.5)
    args = {**inputs(5, 4, 2, 64, 64), **norms(64)}
    args["qkv"][3] = 0
    import gemm_qmv_quantize_gb300 as q
    assert bool(torch.isnan(q.qmv_norm_rope_append(**args, eps=0.0)[3]).all())   # 0 / 0


def test_nan_stays_in_its_head():
    import gemm_qmv_quantize_gb300 as q
    args = {**inputs(3, 4, 2, 64, 64, seed=5), **norms(64)}
    clean = q.qmv_norm_rope_append(**args)
    args["qkv"][1, 64 + 7] = float("nan")
    args["qkv"][2, 3 * 64] = float("inf")
    got = q.qmv_norm_rope_append(**args)
    assert bool(torch.isnan(got[1, 1]).all()) and bool(torch.isnan(got[2, 3, [0, 32]]).all())
    same = torch.ones((3, 4), dtype=torch.bool)
    same[1, 1] = same[2, 3] = False
    assert torch.equal(got[same], clean[same])


def test_indices_outside_are_flagged_and_not_followed():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    args = {**inputs(3, 4, 2, 64, 64, seed=4), **norms(64)}
    args["positions"][0] = torch.tensor([10 ** 9, 5, -1], dtype=torch.int32)
    args["slots"][:] = torch.tensor([0, 1 << 40, 2])
    k0 = args["k_cache"].clone()
    got = q.qmv_norm_rope_append(**args)
    assert q.error_flags(clear=True) == 2
    ends = {**args, "positions": torch.tensor([[299, 5, 0]], dtype=torch.int32, device="cuda"),
            "slots": torch.tensor([0, -1, 2], device="cuda"), "k_cache": k0}
    assert torch.equal(got, q.qmv_norm_rope_append(**ends)) and torch.equal(args["k_cache"], ends["k_cache"])
    assert q.error_flags(clear=True) == 0


def test_empty_and_refusals():
    import gemm_qmv_quantize_gb300 as q
    assert q.qmv_norm_rope_append(**inputs(0, 4, 2, 64, 64), **norms(64)).shape == (0, 4, 64)
    args = {**inputs(2, 4, 2, 64, 64, axes=2), **norms(64)}
    for bad in (dict(q_norm=args["q_norm"][:32].contiguous()), dict(axis_of_pair=[0] * 31),
                dict(qkv=args["qkv"][:, :250].contiguous()), dict(k_norm=norms(128)["k_norm"])):
        with pytest.raises(ValueError):
            q.qmv_norm_rope_append(**{**args, **bad})
    for bad in (dict(q_norm=args["q_norm"].half()), dict(v_cache=args["v_cache"].bfloat16()),
                dict(k_cache=args["k_cache"].float())):
        with pytest.raises(TypeError):
            q.qmv_norm_rope_append(**{**args, **bad})
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(axis_of_pair=[2] * 32)):
        with pytest.raises(q.QmvError):
            q.qmv_norm_rope_append(**{**args, **bad})
