"""GPU tests of what qmv_rope_append_e4m3 does to tokens that a block keeps, for scales that
it does not write itself. Tolerances as in the operator's own tests: kept codes and scales are equal."""
import math

import pytest
import torch

from test_gpu_append_e4m3 import check, inputs, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("slots", [[5], [21, 22, 23], [3, 4, 47, 63, 64, 65], list(range(9, 60))])
@pytest.mark.parametrize("zero", ["k_scale", "v_scale", "both"])
def test_kept_tokens_of_scale_0_stay_0(zero, slots, D):
    """Codes that are not 0 under a scale of 0, as in buffers filled with zeros beside pages that were used before."""
    args = inputs(slots, D=D, seed=len(slots))
    for name in ("k_scale", "v_scale"):
        if zero in (name, "both"):
            args[name].fill_(0)
    first = slots[0]
    kept = args["v_cache"].view(torch.uint8).view(-1, 2, D)[first // 16 * 16:first]
    kept[0, 1, 7] = 0x7f                     # NaN times 0 is NaN
    check(args)
    values = args["k_cache" if zero == "k_scale" else "v_cache"].view(-1, 2, D)[first // 16 * 16:first, 0].float()
    assert bool((values == 0).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -1.0, -math.inf])
def test_kept_tokens_of_no_scale_become_nan(bad):
    args, clean = inputs([20, 21], D=128, seed=3), inputs([20, 21], D=128, seed=3)
    args["k_scale"].fill_(bad)
    args["v_scale"].fill_(bad)
    clean["slots"] -= 4                      # the same rows at a block's start
    clean["positions"] = args["positions"]
    assert torch.equal(run(args), run(clean))
    for name in ("k", "v"):
        got, fresh = (a[name + "_cache"].float().view(-1, 2, 128) for a in (args, clean))
        assert bool(torch.isnan(got[16:20]).all()) and torch.equal(got[20:22], fresh[16:18])
        assert torch.equal(args[name + "_scale"].view(-1, 2)[1], clean[name + "_scale"].view(-1, 2)[1])
        others = torch.cat([args[name + "_scale"].view(-1, 2)[:1], args[name + "_scale"].view(-1, 2)[2:]])
        assert torch.equal(others.nan_to_num(7.0), torch.full_like(others, bad).nan_to_num(7.0))


def test_a_scale_that_does_not_grow_leaves_kept_codes_as_they_are():
    args = inputs([20], seed=4, scale=2.0 ** -30, norm=False)
    before = {n: args[n].clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    check(args)
    for n in ("k_cache", "v_cache"):
        same = torch.arange(128, device="cuda") != 20
        assert torch.equal(args[n].view(torch.uint8).view(128, 2, 64)[same], before[n].view(torch.uint8).view(128, 2, 64)[same])
    for n in ("k_scale", "v_scale"):
        assert torch.equal(args[n], before[n])
