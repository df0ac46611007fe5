"""GPU tests of qmv_paged_attention_e4m3 with NaN codes under scales of 0: value = code * scale is NaN.
Tolerances of what is not NaN as in the operator's own tests."""
import pytest
import torch

from test_gpu_paged_attention_e4m3 import check, inputs, widened

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("long_bound", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("name", ["v", "k"])
def test_nan_codes_of_a_scale_of_0_are_nan(name, T, D, long_bound):
    n = 70
    for token in (3, n - T - 16, n - T, n - 1):           # that all rows see, and that later ones do
        args = inputs(2, T, 6, 2, D, [n, n + 1], 16, seed=41)
        page = int(args["table"][0, token // 16])
        args[name + "_scale"][page] = 0
        args[name + "_cache"].view(torch.uint8)[page, token % 16, 1, 5:9] = 0xff
        got = check(widened(args) if long_bound else args)
        nan = torch.isnan(got)
        first = max(0, token - (n - T))
        assert bool(nan[0, first:, 3:, 5:9 if name == "v" else 64].all()) and not bool(nan[0, :, :3].any() | nan[1].any() | nan[0, :first].any())


@pytest.mark.parametrize("T", [1, 3])
def test_nan_codes_past_the_length_under_a_scale_of_0_are_not_used(T):
    args = inputs(1, T, 4, 2, 128, [37], 16, seed=42)
    page = int(args["table"][0, 2])
    args["v_scale"][page] = 0
    args["v_cache"].view(torch.uint8)[page, 5:] = 0x7f
    assert not bool(torch.isnan(check(args)).any())
