"""GPU tests of qmv_paged_attention_e4m3 against its definition in 64 bits.

Tolerance: the output's rounding (2^-11 or 2^-8 of it, 2^-24 below binary16's normal range);
each term p_j sv_j of the sum over V is rounded to binary16, 2^-11 of it, or 2^-25 of the
row's largest term where it is below the normal range (whole terms are held to 1 at least);
its own error in fp32 (scores up to 2^6 within 2^-22 of themselves and a product of 128 terms within 2^-17 of
the sum of their magnitudes, an exponential) is below 2^-13 of it for the scores drawn here.
"""
import math

import pytest
import torch

import cache8_ref
from cache8_ref import E4M3

pytestmark = pytest.mark.gpu

TYPES = {"f16": (torch.float16, 2.0 ** -11), "bf16": (torch.bfloat16, 2.0 ** -8)}


def inputs(B, T, Hq, Hkv, D, lens, page=16, type_="f16", seed=0, spare=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = max(1, max((n + page - 1) // page for n in lens))
    pages = B * width + spare
    k, ks = cache8_ref.random_cache(g, pages, page, Hkv, D)
    v, vs = cache8_ref.random_cache(g, pages, page, Hkv, D)
    table = torch.randperm(pages, generator=g, device="cuda")[:B * width].to(torch.int32).reshape(B, width).contiguous()
    return dict(q=torch.randn((B, T, Hq, D), generator=g, device="cuda").to(TYPES[type_][0]), k_cache=k, v_cache=v, k_scale=ks,
                v_scale=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def run(args, **kw):
    import gemm_qmv_quantize_gb300 as q
    return q.qmv_paged_attention_e4m3(**args, **kw)


def check(args, type_="f16", scale=None, **kw):
    got = run(args, scale=scale, **kw)
    near(got, args, type_, args["q"].shape[-1] ** -0.5 if scale is None else scale)
    return got


def near(got, args, type_, scale):
    u = TYPES[type_][1]
    o, bound, floor = cache8_ref.attention(args["q"], *(args[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "lens")), scale)
    fine = torch.isfinite(o)
    assert torch.equal(torch.isnan(got), torch.isnan(o))
    err = (got.double() - o).abs()
    tol = u * o.abs() + (2.0 ** -11 + 2.0 ** -13) * bound + 2.0 ** -25 * floor + 2.0 ** -24
    assert bool((err[fine] <= tol[fine]).all()), float((err / tol)[fine].max())


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,page", [
    (1, 1, 1, 1, 64, [1], 16), (1, 1, 8, 1, 128, [16], 16), (2, 1, 32, 8, 128, [17, 560], 16), (3, 1, 40, 8, 128, [0, 300, 1], 32),
    (4, 1, 16, 1, 64, [15, 31, 129, 1000], 64), (2, 5, 8, 2, 64, [5, 777], 32), (3, 2, 10, 2, 128, [1, 2, 333], 16),
    (2, 8, 12, 3, 128, [100, 40], 64), (1, 33, 4, 1, 128, [200], 128), (1, 70, 8, 1, 64, [130], 256), (2, 3, 5, 5, 128, [64, 48], 16),
    (5, 1, 24, 8, 64, [2000, 3, 512, 511, 513], 128), (1, 1, 64, 2, 128, [4097], 64), (1, 4, 3, 1, 128, [3], 16)])
def test_sizes_and_types(B, T, Hq, Hkv, D, lens, page, type_):
    check(inputs(B, T, Hq, Hkv, D, lens, page, type_, seed=B + D), type_)


@pytest.mark.parametrize("lens", [[9000, 1, 4000], [0, 0, 70000]])
def test_long_lengths(lens):
    check(inputs(3, 1, 8, 2, 128, lens, 64, "bf16", seed=1), "bf16")


def test_a_bound_and_a_table_wider_than_the_lengths():
    args = inputs(3, 2, 8, 2, 64, [40, 900, 100], 16, seed=2)
    plain = check(args)
    for max_len in (900, 901, 912):
        check(args, max_len=max_len)
    wide = {**args, "table": torch.cat([args["table"], torch.full_like(args["table"], 10 ** 6)], 1).contiguous()}
    check(wide)          # pages past the lengths are not looked up
    assert plain.shape == args["q"].shape


@pytest.mark.parametrize("T", [1, 4])
def test_what_lies_behind_the_last_token_is_not_used(T):
    lens = [5, 37, 64, 129]
    args = inputs(4, T, 8, 2, 128, lens, 32, seed=3)
    clean = run(args)
    for b, n in enumerate(lens):
        page, at = int(args["table"][b, n // 32]) if n // 32 < args["table"].shape[1] else -1, n % 32
        if page >= 0:
            for name in ("k_cache", "v_cache"):
                args[name].view(torch.uint8)[page, at:] = 0x7f     # NaN
    assert torch.equal(run(args), clean)
    check(args)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,n", [(5, 70), (5, 64), (3, 3), (20, 50), (2, 17)])
def test_nan_of_later_tokens_does_not_reach_earlier_rows(T, n, D):
    """NaN in the newest tokens' keys and values, one at a time, and in several."""
    args = inputs(2, T, 6, 2, D, [n, n + 1], 16, seed=4)
    clean = run(args)
    for token, name, where in ((n - 1, "v_cache", slice(3, 9)), (n - T + 1, "v_cache", slice(0, D)), (n - 1, "k_cache", slice(0, 1))):
        if token < 0:
            continue
        bad = {**args, name: args[name].clone()}
        bad[name].view(torch.uint8)[int(args["table"][0, token // 16]), token % 16, 1, where] = 0xff
        got = check(bad)
        first = max(0, token - (n - T))          # the first of the T tokens that sees it
        assert torch.equal(got[0, :first], clean[0, :first]) and torch.equal(got[1], clean[1])
        assert bool(torch.isnan(got[0, first:, 3:, where if name == "v_cache" else slice(None)]).all())


def widened(args, keys=4096):
    """The same call with a bound of the lengths for which the work is split in runs over all SMs."""
    page, (B, width) = args["k_cache"].shape[1], args["table"].shape
    return {**args, "table": torch.cat([args["table"], args["table"][:, :1].expand(B, max(0, keys // page - width))], 1).contiguous()}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,n", [(5, 70), (5, 64), (3, 3), (20, 500), (2, 1700)])
def test_nan_of_later_tokens_with_a_long_bound(T, n, D):
    args = widened(inputs(3, T, 6, 2, D, [n, n + 1, 4000], 16, seed=4))
    clean = check(args)
    for token, name, where in ((n - 1, "v_cache", slice(3, 9)), (n - T + 1, "v_cache", slice(0, D)), (n - 1, "k_cache", slice(0, 1))):
        if token < 0:
            continue
        bad = {**args, name: args[name].clone()}
        bad[name].view(torch.uint8)[int(args["table"][0, token // 16]), token % 16, 1, where] = 0xff
        got = check(bad)
        first = max(0, token - (n - T))
        assert torch.equal(got[0, :first], clean[0, :first]) and torch.equal(got[1:], clean[1:])
        assert bool(torch.isnan(got[0, first:, 3:, where if name == "v_cache" else slice(None)]).all())


@pytest.mark.parametrize("B,T,Hq,Hkv,D,lens,page,type_", [
    (1, 1, 8, 1, 128, [5], 16, "f16"), (3, 2, 40, 8, 128, [0, 1, 2], 32, "bf16"), (4, 3, 6, 3, 64, [17, 0, 900, 33], 64, "f16"),
    (2, 40, 4, 2, 64, [39, 41], 16, "bf16"), (6, 1, 30, 10, 128, [16, 32, 48, 1, 15, 3000], 16, "f16"), (40, 1, 8, 8, 64, [7] * 39 + [2500], 32, "f16"),
    (300, 1, 2, 1, 128, [30 + i % 90 for i in range(300)], 16, "bf16"), (1, 1, 64, 16, 64, [4096], 256, "f16")])
def test_short_lengths_with_a_long_bound(B, T, Hq, Hkv, D, lens, page, type_):
    check(widened(inputs(B, T, Hq, Hkv, D, lens, page, type_, seed=B + D)), type_)


def test_special_queries_and_lengths_with_a_long_bound():
    args = widened(inputs(3, 4, 4, 2, 64, [0, 2, 4], 16, seed=10))
    got = check(args)
    assert bool((got[0] == 0).all()) and bool((got[1, :2] == 0).all())
    args = widened(inputs(2, 2, 6, 2, 128, [60, 61], 16, seed=11))
    clean = run(args)
    args["q"][0, 1, 2, 7], args["q"][1, 0, 5, 9] = math.nan, math.inf
    got = run(args)
    assert bool(torch.isnan(got[0, 1, 2]).all()) and bool(torch.isnan(got[1, 0, 5]).all())
    got[0, 1, 2], got[1, 0, 5] = clean[0, 1, 2], clean[1, 0, 5]
    assert torch.equal(got, clean)


def test_scales_of_all_sizes():
    """Blocks whose scales are far apart: small values under a large softmax weight and the reverse."""
    args = inputs(2, 1, 8, 2, 128, [400, 90], 16, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    args["v_scale"] = torch.exp2(torch.randint(-64, 40, args["v_scale"].shape, generator=g, device="cuda").float())
    args["k_scale"] = torch.exp2(torch.randint(-20, -6, args["k_scale"].shape, generator=g, device="cuda").float())
    o, bound, floor = cache8_ref.attention(*args.values(), 128 ** -0.5)
    args32 = {**args, "q": args["q"].bfloat16()}
    got = run(args32)
    assert bool(torch.isfinite(got).all())
    o, bound, floor = cache8_ref.attention(*args32.values(), 128 ** -0.5)
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -13) * bound + 2.0 ** -25 * floor
    assert bool(((got.double() - o).abs() <= tol).all())


def test_blocks_of_zero_scale():
    args = inputs(2, 1, 4, 2, 64, [100, 33], 16, seed=7)
    args["v_scale"][::2] = 0
    args["k_scale"][::3] = 0
    check(args)
    args["v_scale"].fill_(0)
    assert bool((check(args) == 0).all())


def test_scales_that_are_no_powers_of_two():
    args = inputs(2, 2, 4, 2, 128, [100, 33], 16, seed=8)
    g = torch.Generator(device="cuda").manual_seed(9)
    for n in ("k_scale", "v_scale"):
        args[n] = torch.rand(args[n].shape, generator=g, device="cuda") * 0.02
    check(args)


def test_rows_without_keys_give_zeros_and_rows_of_minus_infinity_nan():
    args = inputs(3, 4, 4, 2, 64, [0, 2, 4], 16, seed=10)
    got = check(args)
    assert bool((got[0] == 0).all()) and bool((got[1, :2] == 0).all()) and bool((got[1, 2:] != 0).any())
    args = inputs(1, 1, 2, 1, 64, [20], 16, seed=10)
    args["lens"][0] = -5
    assert bool((run(args) == 0).all())
    args["lens"][0] = 20
    args["k_cache"] = torch.ones_like(args["k_cache"].float()).to(E4M3)
    args["q"].zero_()
    args["q"][..., 5] = -math.inf            # every score -inf
    assert bool(torch.isnan(run(args)).all())


def test_nan_and_infinite_queries_stay_in_their_rows():
    for type_ in ("f16", "bf16"):
        args = inputs(2, 2, 6, 2, 128, [60, 61], 16, type_, seed=11)
        clean = run(args)
        args["q"][0, 1, 2, 7] = math.nan
        args["q"][1, 0, 5, 9] = math.inf
        got = run(args)
        assert bool(torch.isnan(got[0, 1, 2]).all()) and bool(torch.isnan(got[1, 0, 5]).all())
        got[0, 1, 2], got[1, 0, 5] = clean[0, 1, 2], clean[1, 0, 5]
        assert torch.equal(got, clean)


def test_large_and_small_bfloat16_queries():
    args = inputs(1, 1, 8, 2, 128, [50], 16, "bf16", seed=12)
    for by, scale in ((2.0 ** 40, 2.0 ** -43.5), (2.0 ** -60, 2.0 ** 56.5), (2.0 ** -130, 2.0 ** 126)):
        scaled = {**args, "q": (args["q"].float() * by).bfloat16()}
        check(scaled, "bf16", scale=scale)


def test_indices_outside_are_flagged_and_not_followed():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    args = inputs(2, 1, 4, 2, 64, [90, 50], 16, seed=13)
    clean = run(args, max_len=90)
    assert q.error_flags(clear=True) == 0
    args["lens"][1] = 10 ** 9
    got = run(args, max_len=90)
    assert q.error_flags(clear=True) == 2 and torch.equal(got[0], clean[0])
    args["lens"][1] = 50
    zero = int(args["table"][0, 2])
    for bad in (-1, args["k_cache"].shape[0], 2 ** 31 - 1):
        args["table"][0, 2] = bad
        got = run(args, max_len=90)
        assert q.error_flags(clear=True) == 2
        args["table"][0, 2] = zero
        zeros = {**args, "k_cache": args["k_cache"].clone(), "v_cache": args["v_cache"].clone()}
        for n in ("k_cache", "v_cache"):
            zeros[n].view(torch.uint8)[zero] = 0
        # Zeros as the definition has them. Not the same bits as a page of zero codes: what the terms of a
        # row's sum are rounded relative to is its largest weight times scale, and a page outside has no
        # scale, so either result is within the tolerance of the value, and of the other within twice that.
        near(got, zeros, "f16", 64 ** -0.5)


def test_offsets_past_32_bits():
    args = inputs(1, 1, 8, 8, 128, [500], 256, seed=14, spare=0)
    few = run(args)
    pages = 17000                                    # 17000 x 256 x 8 x 128 = 4.46e9 codes a cache
    big = dict(args)
    for n in ("k", "v"):
        c = torch.zeros((pages, 256, 8, 128), dtype=torch.uint8, device="cuda")
        s = torch.zeros((pages, 16, 8), device="cuda")
        c[-2:], s[-2:] = args[n + "_cache"].view(torch.uint8), args[n + "_scale"]
        big[n + "_cache"], big[n + "_scale"] = c.view(E4M3), s
    big["table"] = args["table"] + (pages - 2)
    assert torch.equal(run(big), few)


def test_the_same_bits_again_and_on_another_stream_and_in_a_graph():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(5, 1, 40, 8, 128, [3000, 17, 900, 0, 2222], 64, "bf16", seed=15)
    plain = run(args)
    assert torch.equal(run(args), plain)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = run(args, stream=s)
    s.synchronize()
    assert torch.equal(other, plain)
    ws = torch.empty((q.qmv_paged_attention_e4m3_workspace(5, 1, 40, 8, 128, 3008),), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(plain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(args, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain)
    args["lens"].copy_(torch.tensor([5, 1700, 64, 3000, 1], dtype=torch.int32))   # other lengths, the same graph
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run(args))


def test_drawn_sizes():
    import random
    rng = random.Random(20)
    for i in range(25):
        Hkv = rng.choice([1, 2, 3, 8])
        G, D, T, B = rng.randint(1, 9), rng.choice([64, 128]), rng.choice([1, 1, 2, 3, 6]), rng.randint(1, 6)
        lens = [int(2 ** rng.uniform(0, 11)) for _ in range(B)]
        type_ = rng.choice(["f16", "bf16"])
        check(inputs(B, T, G * Hkv, Hkv, D, lens, rng.choice([16, 32, 64, 128, 256]), type_, seed=i), type_)


def test_refusals():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(2, 1, 4, 2, 64, [20, 30], 16, seed=16)
    for bad in (dict(k_scale=args["k_scale"][:2].contiguous()), dict(lens=args["lens"][:1]), dict(table=args["table"].T)):
        with pytest.raises(ValueError):
            run({**args, **bad})
    for bad in (dict(q=args["q"].float()), dict(v_cache=args["v_cache"].view(torch.uint8)), dict(lens=args["lens"].long())):
        with pytest.raises(TypeError):
            run({**args, **bad})
    for kw in (dict(scale=0.0), dict(scale=math.inf), dict(max_len=10 ** 6)):
        with pytest.raises(q.QmvError):
            run(args, **kw)
    with pytest.raises(q.QmvError):
        run({**args, "q": args["q"][:, :, :3].contiguous()})
