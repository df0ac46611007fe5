"""GPU tests of qmv_penalize_logits against its definition in 64 bits.

Tolerance: at most one division or product, one fused penalty (a product and two sums) and
the row's biases for the token, each rounded to fp32: 2^-22 of the largest magnitude that
takes part, per operation. Untouched and masked values are exact.
"""
import math

import pytest
import torch

import decode_ref

pytestmark = pytest.mark.gpu


def inputs(M, V, H, n_bias=0, n_masks=0, seed=0, **off):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = torch.randint(0, H + 1, (M,), generator=g, device="cuda", dtype=torch.int32)
    total[-1] = H
    args = dict(logits=torch.randn((M, V), generator=g, device="cuda") * 4,
                tokens=(V * torch.rand((M, H), generator=g, device="cuda") ** 3).int().clamp_(0, V - 1),
                prompt_len=(total * torch.rand((M,), generator=g, device="cuda")).int(), total_len=total,
                repetition=torch.rand((M,), generator=g, device="cuda") + 0.7,
                presence=torch.randn((M,), generator=g, device="cuda"),
                frequency=torch.randn((M,), generator=g, device="cuda"),
                bias_tokens=None, bias_values=None, mask=None, mask_row=None)
    if n_bias:   # entries repeat and some are unused
        args["bias_tokens"] = torch.randint(-2, min(V, 2 * n_bias), (M, n_bias), generator=g, device="cuda", dtype=torch.int32)
        args["bias_values"] = torch.randn((M, n_bias), generator=g, device="cuda") * 3
    if n_masks:
        args["mask"] = torch.randint(-2 ** 31, 2 ** 31, (n_masks, (V + 31) // 32), generator=g, device="cuda").int()
        args["mask_row"] = torch.randint(-1, n_masks, (M,), generator=g, device="cuda", dtype=torch.int32)
    return {**args, **off}


def check(args, **kw):
    import gemm_qmv_quantize_gb300 as q
    ref = decode_ref.logits(*(args[k] for k in (
        "logits", "tokens", "prompt_len", "total_len", "repetition", "presence", "frequency", "bias_tokens",
        "bias_values", "mask", "mask_row")))
    x = args["logits"].double().cpu().clone()
    big = x.abs().clamp(max=1e30) * 2 + ref.abs().nan_to_num(posinf=0.0) + args["tokens"].shape[1] * 8.0
    if args["bias_values"] is not None:
        big = big + args["bias_values"].double().abs().sum(1, keepdim=True).cpu()
    got = q.qmv_penalize_logits(**args, **kw).cpu()
    fine = torch.isfinite(ref)
    assert torch.equal(got.double()[~fine], ref[~fine])
    seen = ref != x
    assert torch.equal(got.double()[fine & ~seen], ref[fine & ~seen])
    err = (got.double() - ref).abs()
    assert bool((err[fine] <= 2.0 ** -22 * big[fine]).all())
    return got


@pytest.mark.parametrize("M,V,H,n_bias,n_masks", [
    (1, 1, 1, 0, 0), (1, 31, 5, 1, 1), (2, 33, 40, 3, 2), (3, 1000, 0, 0, 0), (4, 8191, 300, 20, 3), (2, 8193, 64, 0, 1),
    (1, 32000, 700, 300, 0), (5, 50257, 1500, 7, 4), (3, 151936, 5000, 40, 2), (40, 1003, 90, 5, 40)])
def test_sizes(M, V, H, n_bias, n_masks):
    check(inputs(M, V, H, n_bias, n_masks, seed=V + M))


@pytest.mark.parametrize("off", ["repetition", "presence", "frequency"])
def test_without_one(off):
    check(inputs(3, 2000, 100, 4, 2, seed=1, **{off: None}))


def test_many_repeats_of_one_token():
    args = inputs(2, 500, 20000, seed=2)
    args["tokens"].fill_(77)
    args["prompt_len"][:] = torch.tensor([0, 19999])
    args["total_len"].fill_(20000)
    check(args)


def test_long_bias_lists_with_repeats():
    args = inputs(2, 3000, 60, 1700, 1, seed=9)      # more entries than a CTA has threads, each token several
    args["bias_tokens"] = args["bias_tokens"].remainder(400)
    check(args)
    check(args, out=args["logits"])


def test_special_values():
    args = inputs(3, 300, 50, 10, 2, seed=3)
    args["logits"][0, :40] = -math.inf
    args["logits"][1, :40] = math.inf
    args["logits"][2, :40] = 0.0
    args["logits"][:, 40:60] = torch.finfo(torch.float32).min / 4
    args["mask_row"][:] = torch.tensor([-1, 0, 1])
    check(args)


def test_everything_masked_and_in_place():
    args = inputs(2, 4001, 30, 5, 2, seed=4)
    args["mask"][0] = 0
    args["mask_row"][:] = torch.tensor([0, 1])
    got = check(args, out=args["logits"])
    assert bool(torch.isneginf(got[0]).all())


def test_nan_stays_where_it_is_allowed():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(1, 64, 8, 0, 1, seed=5)
    args["logits"].fill_(math.nan)
    args["mask"][0, 0], args["mask"][0, 1], args["mask_row"][0] = -1, 0, 0
    got = q.qmv_penalize_logits(**args)[0]
    assert bool(torch.isnan(got[:32]).all()) and bool(torch.isneginf(got[32:]).all())


def test_indices_outside_are_flagged_and_not_followed():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    for name, value in (("tokens", 700), ("total_len", 60), ("mask_row", 9)):
        args = inputs(2, 700, 50, 3, 2, seed=6)
        args["total_len"].fill_(50)
        args["mask_row"][:] = torch.tensor([1, 0])
        (args[name][0] if name == "tokens" else args[name])[0] = value
        check(args)
        assert q.error_flags(clear=True) == 2, name
    args = inputs(2, 700, 50, 3, 2, seed=6)
    args["tokens"][:, ::3] = -1                       # skipped, as padding
    check(args)
    assert q.error_flags(clear=True) == 0


def test_refusals():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(2, 100, 10, 3, 2, seed=7)
    with pytest.raises(TypeError):
        q.qmv_penalize_logits(**{**args, "logits": args["logits"].half()})
    with pytest.raises(ValueError):
        q.qmv_penalize_logits(**{**args, "mask": args["mask"][:, :3].contiguous()})
    with pytest.raises(ValueError):
        q.qmv_penalize_logits(**{**args, "bias_values": None})
    with pytest.raises(ValueError):
        q.qmv_penalize_logits(**{**args, "tokens": args["tokens"].T})
    with pytest.raises(q.QmvError):
        q.qmv_penalize_logits(**{**args, "mask": args["mask"][:1].contiguous(), "mask_row": None})   # a mask a row


@pytest.mark.parametrize("at", [0, 511, 512, 699])
def test_bias_tokens_outside_are_flagged_and_not_followed(at):
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    args = inputs(2, 9000, 50, 700, 2, seed=8)
    args["bias_tokens"][1, at] = 8999
    check(args)
    assert q.error_flags(clear=True) == 0
    for token in (9000, 2 ** 31 - 1):
        args["bias_tokens"][1, at] = token
        check(args)
        assert q.error_flags(clear=True) == 2
