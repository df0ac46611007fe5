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
from test_gpu_paged_attention_e4m3 import TYPES, inputs, run, widened

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
