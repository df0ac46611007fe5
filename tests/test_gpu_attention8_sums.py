"""GPU tests of what qmv_paged_attention_e4m3 holds of the sums over V, closer than binary16's
steps, and of the ends of the scales' range.

Tolerance of an output o = (sum_j p_j V_j) / (sum_j p_j), with the sum of magnitudes bound = sum_j p_j |V_j|: its
own rounding, half a step of the type (2^-25 below binary16's normal range); a score's error in fp32, at
most D / 16 + 2 = 10 additions to a sum, each within 2^-22 of the magnitudes' sum, so 2^-18 of c sum_i |q_i K_i|, in
a term and, at most as much, in the denominator; exponentials and the terms' two parts, 2^-20 together; a
warp's additions of blocks, at most 40 here, 2^-22 each in either sum, 2^-15.7 together.
"""
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
