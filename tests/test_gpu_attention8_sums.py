"""GPU tests of what qmv_paged_attention_e4m3 holds of the sums over V, closer than binary16's
steps, and of the ends of the scales' range.

Tolerance of an output o = (sum_j p_j V_j) / (sum_j p_j), with the sum of magnitudes bound = sum_j p_j |V_j|: its
own rounding, half a step of the type (2^-25 below binary16's normal range); a score's error in fp32, at
most D / 16 + 2 = 10 additions to a sum, each within 2^-22 of the magnitudes' sum, so 2^-18 of c sum_i |q_i K_i|, in
a term and, at most as much, in the denominator; exponentials and the terms' two parts, 2^-20 together; a
warp's additions of blocks, at most 40 here, 2^-22 each in either sum, 2^-15.7 together.
"""
import math

import pytest
import torch

import cache8_ref
from cache8_ref import E4M3
from test_gpu_paged_attention_e4m3 import TYPES, inputs, near, run, widened

pytestmark = pytest.mark.gpu


def check(args, type_, scale, most_score):
    """most_score: of c sum_i |q_i K_i|."""
    got = run(args, scale=scale).double()
    o, bound, _ = cache8_ref.attention(*(args[n] for n in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "table", "lens")), scale)
    tol = TYPES[type_][1] * o.abs() + (2.0 ** -25 if type_ == "f16" else 0.0) + (2.0 ** -17 * most_score + 2.0 ** -15) * bound
    worst = float(((got - o).abs() / tol.clamp(min=1e-300)).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("long_bound", [False, True])
@pytest.mark.parametrize("D,T,G", [(64, 1, 8), (128, 1, 5), (128, 3, 5), (64, 9, 3), (128, 1, 16)])
def test_terms_are_held_closer_than_binary16(D, T, G, long_bound):
    """Softmaxes that are nearly flat, over few keys, and values of both signs: what a term rounded to 2^-11 would leave
    shows in outputs that are small for the magnitudes in them."""
    lens = [T + 1, T + 16, 60, 200]
    args = inputs(4, T, 2 * G, 2, D, lens, 32, seed=D + T + G)
    args["k_scale"].fill_(2.0 ** -10)
    if long_bound:
        args = widened(args)
    k = cache8_ref.values(args["k_cache"], args["k_scale"]).abs().amax(dim=(0, 1, 2))   # [D]
    most = float((args["q"].double().abs() @ k).max()) * D ** -0.5
    check(args, "f16", D ** -0.5, most)


def close(got, args, scale):
    """bfloat16 outputs of any size: half a step, and the terms' errors as above with scores of magnitude 2^5 at most."""
    o, bound, _ = cache8_ref.attention(*(args[n] for n in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "table", "lens")), scale)
    assert bool((o != 0).any()) and bool(((got.double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -12 + 2.0 ** -15) * bound).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("exponent", [-80, -64, 90])
def test_ends_of_the_scales_range(exponent, D):
    for lens in ([600, 17], [600, 4000]):        # by clusters, and in runs
        args = inputs(2, 1, 8, 2, D, lens, 16, "bf16", seed=31)
        args["k_scale"].fill_(2.0 ** -9)
        args["v_scale"].fill_(2.0 ** exponent)
        close(run(args), args, D ** -0.5)


@pytest.mark.parametrize("small", [2.0 ** -81, 2.0 ** -90, 2.0 ** -100, 1e-45, -1.0, float("-inf"), float("nan")])
def test_scales_that_count_as_0(small):
    """Of values, those below the range and no scales at all; of keys, the latter."""
    for lens in ([600, 17], [600, 4000]):
        args = inputs(2, 2, 8, 2, 128, lens, 16, "bf16", seed=32)
        args["v_scale"][::3] = 0
        if not small > 0:
            args["k_scale"][::2] = 0
        expected = run(args)
        args["v_scale"][::3] = small
        if not small > 0:
            args["k_scale"][::2] = small
        assert torch.equal(run(args), expected)
        args["v_scale"].fill_(small)
        assert bool((run(args) == 0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("weight,code,n", [(18.0, 448.0, 4001), (18.0, 448.0, 200), (20.0, 448.0, 9000)])
def test_many_light_terms_beside_a_heavy_one(weight, code, n, D):
    """The first key weighs e^18 or e^20 (2^26, 2^29) times what each other one does and has values of 0: the outputs
    are the others', none of which is dropped for being light: a term is within 2^-32 of the largest, half of binary16's least
    step for the 2^7 that the largest is at least."""
    args = inputs(1, 1, 2, 1, D, [n], 16, seed=33)
    for name in ("k_cache", "v_cache"):
        args[name].view(torch.uint8).zero_()
    for name in ("k_scale", "v_scale"):
        args[name].fill_(1.0)
    at = int(args["table"][0, 0])
    args["q"].zero_()
    args["q"][..., 0] = 1.0
    args["k_cache"][at, 0, 0, 0] = weight
    args["v_cache"].copy_(torch.full_like(args["v_cache"].float(), code).to(E4M3))
    args["v_cache"].view(torch.uint8)[at, 0].zero_()
    got = run(args, scale=1.0).double()
    o = cache8_ref.attention(*(args[n_] for n_ in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "table", "lens")), 1.0)[0]
    step = 2.0 ** -32 * math.exp(weight)     # of a term
    assert bool(((got - o).abs() <= (2.0 ** -11 + 2.0 ** -15 + step) * o + 2.0 ** -25).all()), (float(got.min()), float(o.min()))


def long_runs(B, Hq, Hkv, D, lens, pages, type_="f16", T=1, seed=61):
    """Requests over a few pages again and again, so many of them that a run is a request's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    args = inputs(1, T, Hq, Hkv, D, [256 * pages], 256, type_, seed=seed, spare=0)
    width = (max(lens) + 255) // 256
    args["table"] = torch.randint(0, pages, (B, width), generator=g, device="cuda", dtype=torch.int32)
    args["q"] = torch.randn((B, T, Hq, D), generator=g, device="cuda").to(args["q"].dtype)
    args["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return args


@pytest.mark.parametrize("D,Hq,B", [(128, 8, 152), (128, 128, 152), (64, 8, 304)])
def test_long_sums_of_one_sign_are_not_cut(D, Hq, B):
    """4096 blocks a run, values that are all positive: what the products truncate adds up in one direction (4e-4 of the
    outputs). The mean over 1024 and more outputs of (got - o) / o: each output's rounding is within 2^-11 and of either
    sign, so the mean's is within 2^-11 / 32 but for 1 in 10^3; a part of 512 blocks is at most 1024 truncations of 2^-24, half
    of that in the mean, too small: 2^-15; sums in fp32, 2^-17."""
    args = long_runs(B, Hq, 8, D, [65536] * B, 4)
    args["table"] = (torch.arange(256, device="cuda", dtype=torch.int32) % 4).expand(B, 256).contiguous()
    args["q"] = args["q"][:1].expand(B, 1, Hq, D).contiguous()
    args["k_scale"].fill_(2.0 ** -10)
    args["v_cache"] = args["v_cache"].float().abs().to(E4M3)
    o, bound, _ = cache8_ref.attention(args["q"][:1], args["k_cache"], args["v_cache"], args["k_scale"], args["v_scale"], args["table"][:1],
                                       torch.tensor([1024]), D ** -0.5)
    off = (run(args).double() - o) / o
    assert float(off.abs().max()) <= 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -15
    assert abs(float(off.mean())) <= 2.0 ** -16 + 2.0 ** -15 + 2.0 ** -17, float(off.mean())


@pytest.mark.parametrize("T,Hq,type_,D", [(1, 8, "f16", 128), (3, 8, "bf16", 128), (2, 64, "f16", 128), (2, 8, "bf16", 64), (3, 64, "f16", 64)])
def test_runs_of_several_parts(T, Hq, type_, D):
    """Lengths about two parts and more of 512 blocks, scales that differ from page to page, and NaN in a newest token."""
    B = 160 if D == 128 else 320
    args = long_runs(B, Hq, 8, D, [17000 - 53 * (b % 160) for b in range(B)], 96, type_, T, seed=62)
    g = torch.Generator(device="cuda").manual_seed(63)
    for n in ("k_scale", "v_scale"):
        args[n] = torch.exp2(torch.randint(-11, -4, args[n].shape, generator=g, device="cuda").float())
    n = int(args["lens"][7])
    own, at = args["table"][7].tolist(), (n - 1) // 256
    got = run(args)
    some = [0, 7, 80, B - 1]
    near(got[some], {k: v[some].contiguous() if k in ("q", "table", "lens") else v for k, v in args.items()}, type_, D ** -0.5)
    if T > 1:                                       # a page of request 7's own, with NaN in its newest token
        for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
            args[name] = torch.cat([args[name].view(torch.uint8), args[name].view(torch.uint8)[own[at]:own[at] + 1]]).view(args[name].dtype)
        args["table"][7, at] = 96
        args["v_cache"].view(torch.uint8)[96, (n - 1) % 256, 2, 9] = 0x7f
        bad = run(args)
        G = Hq // 8
        assert bool(torch.isnan(bad[7, T - 1, 2 * G:3 * G, 9]).all()) and int(torch.isnan(bad).sum()) == G
        assert torch.equal(torch.where(torch.isnan(bad), got, bad), got)
