"""GPU tests of qmv_rope_append_e4m3 against its definition in 64 bits.

Tolerance of a code: half a step of E4M3 (2^-4 of the value, 2^-10 scales below 2^-6 scales),
and the value's own error before it is rounded, 2^-20 times twice the largest normed value (see the norms'
tests); v is not computed, so its codes are equal to the conversion's, as are the scales and
the codes of tokens that were there before.
"""
import math

import pytest
import torch

import cache8_ref
from cache8_ref import E4M3

pytestmark = pytest.mark.gpu


def inputs(slots, Hq=4, Hkv=2, D=64, rot=None, axes=1, page=16, pages=8, norm=True, seed=0, scale=1.0):
    import gemm_qmv_quantize_gb300 as q
    g = torch.Generator(device="cuda").manual_seed(seed)
    rot, M = D if rot is None else rot, len(slots)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k, ks = cache8_ref.random_cache(g, pages, page, Hkv, D)
    v, vs = cache8_ref.random_cache(g, pages, page, Hkv, D)
    return dict(qkv=r(M, (Hq + 2 * Hkv) * D) * scale,
                positions=torch.randint(0, 300, (axes, M), generator=g, device="cuda", dtype=torch.int32),
                table=q.qmv_rope_table(300, rot, 10000.0, "cuda"), axis_of_pair=[i % axes for i in range(rot // 2)],
                slots=torch.tensor(slots, dtype=torch.int64, device="cuda"), k_cache=k, v_cache=v, k_scale=ks, v_scale=vs,
                q_norm=r(D) if norm else None, k_norm=r(D) + 1 if norm else None)


def run(args, **kw):
    import gemm_qmv_quantize_gb300 as q
    return q.qmv_rope_append_e4m3(**args, **kw)


def check(args, eps=1e-6, interleaved=False, u=2.0 ** -11, **kw):
    Hkv, D = args["k_cache"].shape[2:]
    before = {n: args[n].clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    got = run(args, eps=eps, interleaved=interleaved, **kw)
    qr, kr, vr = cache8_ref.heads(args["qkv"], args["positions"], args["table"], args["axis_of_pair"], Hkv, D, interleaved,
                                  args["q_norm"], args["k_norm"], eps)
    finite = lambda t: float(t[torch.isfinite(t)].abs().max()) if bool(torch.isfinite(t).any()) else 0.0  # noqa: E731
    off = 2.0 ** -19 * 1.5 * max(finite(qr), finite(kr))
    fine = torch.isfinite(qr)
    assert bool(((got.double() - qr).abs()[fine] <= (u * qr.abs() + off + 2.0 ** -25)[fine]).all())
    assert bool(torch.isnan(got[torch.isnan(qr)]).all())
    for name, new, err in (("k", kr, off), ("v", vr, 0.0)):
        codes, scale, wanted = cache8_ref.append(new, args["slots"], before[name + "_cache"], before[name + "_scale"])
        assert torch.equal(args[name + "_scale"].double().reshape(scale.shape), scale), name
        have = args[name + "_cache"].double().reshape(codes.shape)
        s = scale.repeat_interleave(16, 0)[:, :, None]
        is_new = torch.isnan(codes).all(-1).all(-1)
        assert torch.equal(have[~is_new].nan_to_num(1e9), codes[~is_new].nan_to_num(1e9)), name   # as they were, or moved
        want, s = wanted[is_new], s.expand_as(codes)[is_new]
        nan = torch.isnan(want)
        assert bool(torch.isnan(have[is_new][nan]).all()), name
        if err == 0.0:
            assert torch.equal(have[is_new][~nan], (want / s)[~nan].float().to(E4M3).double()), name
        step = (want.abs() * 2.0 ** -4).maximum(s * 2.0 ** -10) + err
        assert bool(((have[is_new] * s - want).abs()[~nan] <= step[~nan]).all()), name
    return got


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("slots,kw", [
    ([0], {}), ([5], {}), ([15], dict(D=128)), (list(range(16)), dict(D=128)), (list(range(3, 90)), {}),
    (list(range(37, 96)) + list(range(4, 9)) + [97] + [17], dict(D=128, Hq=10, Hkv=5, page=32)),
    ([33, 34, -1, -1, 64, 65, 66], dict(rot=32)), ([20, 127, 0, 50, 111], dict(D=128, rot=64, axes=3, Hq=16, Hkv=16)),
    (list(range(16, 48)), dict(rot=0)), ([64 + i for i in range(64)], dict(page=64, Hq=1, Hkv=1)),
    ([250 + i for i in range(40)], dict(page=256, pages=2, Hq=9, Hkv=9))])
def test_slots_sizes_and_types(slots, kw, interleaved, dtype):
    args = inputs(slots, **kw, seed=len(slots))
    check(args, interleaved=interleaved, dtype=dtype, u=2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8)


@pytest.mark.parametrize("D", [64, 128])
def test_a_sequence_token_by_token(D):
    """Every step against the definition: scales grow with the tokens, codes of the block follow."""
    args = inputs([0], D=D, norm=False, seed=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    for slot in range(16, 16 + 40):
        args["slots"][0] = slot
        args["qkv"] = torch.randn(args["qkv"].shape, generator=g, device="cuda") * 2.0 ** ((slot * 7) % 19 - 9)
        check(args)


def test_what_was_in_a_block_that_starts_is_forgotten():
    args = inputs([32], seed=4)
    args["k_scale"].fill_(2.0 ** 100)
    args["v_scale"].fill_(float("nan"))
    run(args)
    assert bool((args["k_scale"].view(-1, 2)[2] < 1).all()) and bool((args["v_scale"].view(-1, 2)[2] < 1).all())
    assert bool((args["k_scale"].view(-1, 2)[3] == 2.0 ** 100).all())


def test_the_largest_value_meets_448():
    for largest, scale in ((448.0, 1.0), (448.0 * (1 + 2.0 ** -23), 2.0), (447.9, 1.0), (0.875, 2.0 ** -9), (0.8750001, 2.0 ** -8),
                           (3.4e38, 2.0 ** 120), (1e-45, 2.0 ** -64), (0.0, 2.0 ** -64)):
        args = inputs([16], norm=False, rot=0)
        args["qkv"] *= 0
        args["qkv"][0, -1] = largest     # of the last v head
        args["v_scale"].fill_(2.0 ** -60)
        check(args)
        assert float(args["v_scale"].view(-1, 2)[1, 1]) == scale, largest


def test_nan_and_infinities_become_nan_and_move_no_scale():
    args = inputs(list(range(16, 26)), norm=False, rot=0, seed=6)
    args["qkv"][3, -5:] = torch.tensor([math.nan, math.inf, -math.inf, 1.0, -2.0], device="cuda")
    args["qkv"][7, 4 * 64:5 * 64] = math.inf
    check(args)
    codes = args["v_cache"].view(-1, 2, 64)[19, 1, -5:].float()
    assert bool(torch.isnan(codes[:3]).all()) and not bool(torch.isnan(codes[3:]).any())
    args["slots"] = args["slots"][:1] + 10
    args = {**args, "qkv": args["qkv"][:1] * 1000, "positions": args["positions"][:, :1].contiguous()}
    check(args)                           # codes that are NaN stay so when the scale grows
    assert bool(torch.isnan(args["v_cache"].view(-1, 2, 64)[19, 1, -5:-2].float()).all())


def test_all_padding_and_empty():
    args = inputs([-1, -7, -1], seed=7)
    check(args)
    args = inputs([], seed=8)
    assert run(args).shape == (0, 4, 64)


def test_indices_outside_are_flagged_and_not_followed():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    args = inputs([127, 128, 1 << 40, 3], seed=9)   # 8 pages of 16
    check(args)
    assert q.error_flags(clear=True) == 2
    args = inputs([1, 2, 3], seed=9)
    args["positions"][0] = torch.tensor([10 ** 9, 5, -1], dtype=torch.int32)
    ends = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in args.items()}
    ends["positions"][0] = torch.tensor([299, 5, 0], dtype=torch.int32)
    assert torch.equal(run(args), run(ends)) and torch.equal(args["k_cache"].view(torch.uint8), ends["k_cache"].view(torch.uint8))
    assert q.error_flags(clear=True) == 2


def test_the_same_call_twice_gives_the_same():
    args = inputs(list(range(5, 70)), D=128, seed=10)
    first = run(args)
    codes, scale = args["k_cache"].clone(), args["k_scale"].clone()
    assert torch.equal(run(args), first)
    assert torch.equal(args["k_cache"].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(args["k_scale"], scale)


def test_slots_past_32_bits_of_bytes():
    args = inputs([0, 1, 2], D=128, Hkv=8, Hq=8, norm=False, seed=11)
    pages, page = 17000, 256                          # 17000 x 256 x 8 x 128 = 4.46e9 codes a cache
    far = (pages - 1) * page + 13
    big = {**args, "slots": args["slots"] + far}
    for n in ("k", "v"):
        big[n + "_cache"] = torch.zeros((pages, page, 8, 128), dtype=torch.uint8, device="cuda").view(E4M3)
        big[n + "_scale"] = torch.full((pages, page // 16, 8), 2.0 ** -7, device="cuda")
    run(big)
    near = {**big, "slots": args["slots"] + 13}
    for n in ("k", "v"):
        near[n + "_cache"] = torch.zeros((1, page, 8, 128), dtype=torch.uint8, device="cuda").view(E4M3)
        near[n + "_scale"] = torch.full((1, page // 16, 8), 2.0 ** -7, device="cuda")
    run(near)
    for n in ("k", "v"):
        assert torch.equal(big[n + "_cache"].view(torch.uint8)[-1], near[n + "_cache"].view(torch.uint8)[0])
        assert torch.equal(big[n + "_scale"][-1], near[n + "_scale"][0])
        assert not bool(big[n + "_cache"].view(torch.uint8)[:-1].any())


def test_refusals():
    import gemm_qmv_quantize_gb300 as q
    args = inputs([1, 2], seed=12)
    for bad in (dict(k_scale=args["k_scale"][:1].contiguous()), dict(q_norm=args["q_norm"][:8].contiguous())):
        with pytest.raises(ValueError):
            run({**args, **bad})
    for bad in (dict(k_cache=args["k_cache"].view(torch.uint8)), dict(v_scale=args["v_scale"].half())):
        with pytest.raises(TypeError):
            run({**args, **bad})
    with pytest.raises(TypeError):
        run(args, dtype=torch.float32)
    with pytest.raises(q.QmvError):
        run(inputs([1], D=96))
    with pytest.raises(ValueError):
        run(inputs([1], page=8))
