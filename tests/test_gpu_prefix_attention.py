"""GPU tests of qmv_prefix_attention against its definition in 64 bits.

Tolerance, from the arithmetic, with u = 2^-11 (binary16) or 2^-8 (bfloat16) and
bound = sum_j p_j |V_j|: a probability is rounded once to the 16-bit type before the
product with V (u bound); a score is an fp32 sum of at most 128 exact products, within
128 x 2^-23 of the sum of their absolute values, below 128 x 2^-23 x 60 ~ 1e-3 at these
inputs (|q . k| sums below 60 after scaling), which moves a probability by as much
(1e-3 bound, and as much again through the sum of all); the output is rounded once
(u |o|, 2^-24 below binary16's normal range).
"""
import math
import random

import pytest
import torch

import decode_ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": (torch.float16, 2.0 ** -11), "bf16": (torch.bfloat16, 2.0 ** -8)}


def inputs(B, T, Hq, Hkv, D, prefix, own_len, page=16, type_="f16", seed=0, own_pages=None, q_scale=1.0):
    """Pages in no order; everything past a length, and every page unused, is NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[type_][0]
    n_prefix = (prefix + page - 1) // page
    if own_pages is None:
        own_pages = max([(n + page - 1) // page for n in own_len] + [1])
    pages = n_prefix + B * own_pages + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    k, v = (torch.full((pages, page, Hkv, D), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    prefix_table = order[:n_prefix].contiguous()
    own_table = order[n_prefix:n_prefix + B * own_pages].reshape(B, own_pages).contiguous()
    for table, n in [(prefix_table, prefix)] + [(own_table[b], own_len[b]) for b in range(B)]:
        for j in range(0, n, page):
            m = min(page, n - j)
            p = int(table[j // page])
            for c in (k, v):
                c[p, :m] = torch.randn((m, Hkv, D), generator=g, device="cuda").to(dtype)
    return dict(q=(torch.randn((B, T, Hq, D), generator=g, device="cuda") * q_scale).to(dtype), k_cache=k, v_cache=v,
                prefix_table=prefix_table, prefix_len=prefix, own_table=own_table,
                own_len=torch.tensor(own_len, dtype=torch.int32, device="cuda"))


def check(args, type_, scale=None, **kw):
    import gemm_qmv_quantize_gb300 as q
    D = args["q"].shape[3]
    ref, bound = decode_ref.attention(**args, scale=1 / math.sqrt(D) if scale is None else scale)
    got = q.qmv_prefix_attention(**args, scale=scale, **kw)
    u = TYPES[type_][1]
    tol = u * ref.abs() + (u + 2e-3) * bound + 2.0 ** -24
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).nan_to_num(1e9).max())
    return got


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,prefix,own_len,page", [
    (1, 1, 1, 1, 64, 1, [0], 16), (1, 1, 1, 1, 128, 0, [1], 16), (1, 1, 8, 2, 128, 127, [3], 16),
    (2, 1, 8, 2, 128, 128, [1, 128], 32), (3, 1, 7, 1, 64, 129, [17, 0, 300], 64), (2, 1, 40, 8, 128, 1000, [5, 33], 64),
    (4, 2, 12, 4, 64, 513, [2, 1, 0, 140], 16), (2, 8, 10, 2, 128, 260, [8, 100], 128), (1, 5, 6, 6, 64, 77, [40], 256),
    (19, 1, 14, 2, 128, 700, [1 + 13 * i for i in range(19)], 16), (33, 3, 8, 2, 64, 385, [3 + i for i in range(33)], 32)])
def test_sizes_types_pages(B, T, Hq, Hkv, D, prefix, own_len, page, type_):
    check(inputs(B, T, Hq, Hkv, D, prefix, own_len, page, type_, seed=prefix + B), type_)


@pytest.mark.parametrize("prefix", [2000, 4096 + 63])
def test_long_prefix_split_over_the_device(prefix):
    check(inputs(6, 1, 8, 2, 128, prefix, [9, 600, 0, 1, 129, 255], 64, "bf16", seed=1), "bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv,prefix,own_len", [
    (20, 1, 8, 2, 1500, [3 * i for i in range(20)]), (2, 20, 8, 2, 515, [300, 20]), (9, 4, 9, 1, 1100, [4 + 60 * i for i in range(9)])])
def test_pages_longer_than_a_tile(B, T, Hq, Hkv, D, prefix, own_len):
    check(inputs(B, T, Hq, Hkv, D, prefix, own_len, 256, "bf16", seed=B), "bf16")


@pytest.mark.parametrize("seed", range(20))
def test_drawn_sizes(seed):
    rng = random.Random(seed)
    Hkv, G, D, T = rng.choice([1, 2, 3]), rng.randint(1, 9), rng.choice([64, 128]), rng.choice([1, 1, 2, 4, 11])
    B = rng.choice([1, 2, 7, 30, 70])
    most = rng.choice([0, 1, 40, 300]) if B > 7 else rng.choice([1, 200, 1500])
    own_len = [rng.randint(0, most) for _ in range(B)]
    prefix = rng.choice([0, 1, 63, 128, 129, 400, 2200])
    type_ = rng.choice(["f16", "bf16"])
    check(inputs(B, T, Hkv * G, Hkv, D, prefix, own_len, rng.choice([16, 32, 64, 128, 256]), type_, seed=seed), type_)


def test_more_rows_than_a_tile():
    # 48 requests x 2 tokens x 5 heads = 480 rows over one key head
    check(inputs(48, 2, 5, 1, 128, 300, [2 + i for i in range(48)], 32, "f16", seed=2), "f16")


@pytest.mark.parametrize("type_,B,T,Hq,Hkv,D,prefix,own_len,page", [
    ("f16", 2, 10, 8, 1, 128, 200, [10, 333], 16),        # 80 rows of a request and key head
    ("bf16", 3, 40, 5, 1, 64, 129, [40, 7, 300], 32),     # 200 rows
    ("bf16", 2, 70, 8, 1, 128, 0, [70, 200], 64),         # 560 rows, no prefix
    ("f16", 1, 17, 8, 2, 128, 640, [1000], 128),
    ("f16", 2, 16, 4, 1, 64, 0, [0, 40], 16)])            # 64 rows: the few-rows kernel's most
def test_many_tokens_of_a_request(type_, B, T, Hq, Hkv, D, prefix, own_len, page):
    check(inputs(B, T, Hq, Hkv, D, prefix, own_len, page, type_, seed=T), type_)


@pytest.mark.parametrize("type_,B,T,Hq,Hkv,D,prefix,own_len,page", [
    ("f16", 2, 1, 8, 2, 128, 5001, [0, 30], 16), ("bf16", 1, 2, 8, 1, 64, 3333, [40], 64),
    ("bf16", 16, 1, 2, 2, 128, 1025, [i for i in range(16)], 256), ("f16", 3, 1, 7, 1, 64, 200, [0, 0, 0], 32)])
def test_few_rows_behind_a_prefix(type_, B, T, Hq, Hkv, D, prefix, own_len, page):
    check(inputs(B, T, Hq, Hkv, D, prefix, own_len, page, type_, seed=prefix), type_)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_long_own_keys_in_ranges(type_, D):
    check(inputs(2, 2, 6, 2, D, 70, [3001, 1500], 16, type_, seed=11), type_)


def test_rows_without_a_key_are_zero():
    args = inputs(3, 4, 4, 2, 64, 0, [0, 2, 5], 16)
    got = check(args, "f16")
    assert not got[0].any() and not got[1, :2].any() and got[1, 2:].any()
    none = inputs(2, 1, 4, 2, 64, 0, [0, 0], 16)
    assert not check(none, "f16").any()
    assert not check(none, "f16", max_own=0).any()


def test_one_key_is_its_value():
    args = inputs(2, 1, 4, 2, 128, 0, [1, 1], 16, q_scale=30.0)
    got = check(args, "f16")
    v = torch.stack([args["v_cache"][int(args["own_table"][b, 0]), 0] for b in range(2)])
    assert torch.equal(got[:, 0], v.repeat_interleave(2, 1))


@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_growing_scores(type_):
    """Scores that rise along the keys: the running maximum moves at every step."""
    args = inputs(2, 1, 4, 1, 64, 640, [100, 40], 16, type_, seed=3)
    for table, n in [(args["prefix_table"], 640)] + [(args["own_table"][b], int(args["own_len"][b])) for b in (0, 1)]:
        for j in range(n):
            args["k_cache"][int(table[j // 16]), j % 16] = (0.02 * j) * torch.ones((1, 64), device="cuda")
    args["q"] = torch.ones_like(args["q"])
    check(args, type_, scale=1 / 8)


def test_large_scores_and_scales():
    check(inputs(2, 1, 4, 2, 128, 300, [20, 7], 16, seed=4, q_scale=6.0), "f16", scale=0.05)
    check(inputs(2, 1, 4, 2, 128, 300, [20, 7], 16, seed=4), "f16", scale=1e-3)


def test_wide_tables_and_bounds():
    args = inputs(3, 1, 4, 2, 64, 100, [5, 60, 0], 16, own_pages=40)
    args["own_table"][:, 4:] = 2 ** 31 - 1            # never looked at
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    a, b = check(args, "f16", max_own=60), check(args, "f16")
    assert (a.float() - b.float()).abs().max() < 1e-2
    assert q.error_flags(clear=True) == 0


def test_indices_outside_are_flagged_and_not_followed():
    import gemm_qmv_quantize_gb300 as q
    q.error_flags(clear=True)
    args = inputs(2, 1, 4, 2, 64, 100, [5, 60], 16, seed=7)
    args["own_table"][0, 0] = 2 ** 30
    args["prefix_table"][3] = -5
    q.qmv_prefix_attention(**args)
    assert q.error_flags(clear=True) == 2
    args = inputs(2, 1, 4, 2, 64, 100, [5, 60], 16, seed=7)
    cut = q.qmv_prefix_attention(**{**args, "own_len": torch.tensor([5, 7], dtype=torch.int32, device="cuda")}, max_own=7)
    assert q.error_flags(clear=True) == 0
    assert torch.equal(cut, q.qmv_prefix_attention(**args, max_own=7))
    assert q.error_flags(clear=True) == 2


def test_same_call_same_bits_and_other_streams():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(5, 1, 8, 2, 128, 3000, [30, 1, 400, 0, 77], 64, "bf16", seed=5)
    first = q.qmv_prefix_attention(**args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = torch.empty_like(first)
    q.qmv_prefix_attention(**args, out=second, stream=s)
    with torch.cuda.stream(s):
        third = q.qmv_prefix_attention(**args)
    s.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)


def test_cache_whose_offsets_pass_32_bits():
    """2^16 pages x 64 x 8 x 128 elements: the last pages lie past 2^32 elements."""
    page, Hkv, D, pages = 64, 8, 128, 65538
    k, v = (torch.zeros((pages, page, Hkv, D), dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.tensor([pages - 1, 0, pages - 2], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    for p in table.tolist():
        for c in (k, v):
            c[p] = torch.randn((page, Hkv, D), generator=g, device="cuda").half()
    q_ = torch.randn((1, 1, 16, D), generator=g, device="cuda").half()
    args = dict(q=q_, k_cache=k, v_cache=v, prefix_table=table[:2].contiguous(), prefix_len=100,
                own_table=table[2:].reshape(1, 1).contiguous(), own_len=torch.tensor([50], dtype=torch.int32, device="cuda"))
    check(args, "f16")


def test_refusals():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(2, 1, 4, 2, 64, 100, [5, 60], 16)
    for bad in (dict(max_own=65), dict(scale=0.0), dict(scale=math.inf), dict(scale=-1.0)):
        with pytest.raises(q.QmvError):
            q.qmv_prefix_attention(**args, **bad)
    with pytest.raises(q.QmvError):
        q.qmv_prefix_attention(**inputs(1, 1, 4, 2, 80, 20, [5], 16))      # head size
    with pytest.raises(q.QmvError):
        q.qmv_prefix_attention(**inputs(1, 1, 3, 2, 64, 20, [5], 16))      # heads that do not divide
    with pytest.raises(q.QmvError):
        q.qmv_prefix_attention(**inputs(1, 1, 4, 2, 64, 20, [5], 24))      # page size
    with pytest.raises(ValueError):
        q.qmv_prefix_attention(**{**args, "prefix_len": 113})              # more keys than pages
    with pytest.raises(TypeError):
        q.qmv_prefix_attention(**{**args, "q": args["q"].bfloat16()})
    with pytest.raises(TypeError):
        q.qmv_prefix_attention(**{**args, "own_len": args["own_len"].long()})


def check_special(args, type_, **kw):
    """check, where inputs that are used hold infinities and NaN: those of the result are the definition's."""
    import gemm_qmv_quantize_gb300 as q
    D = args["q"].shape[3]
    ref, bound = decode_ref.attention(**args, scale=1 / math.sqrt(D))
    got = q.qmv_prefix_attention(**args, **kw).double()
    u = TYPES[type_][1]
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
    assert bool(((got - ref).abs() <= u * ref.abs() + (u + 2e-3) * bound + 2.0 ** -24)[fine].all())
    return got


def own_place(args, b, key):
    """(page, offset) of an own key of request b."""
    page = args["k_cache"].shape[1]
    return int(args["own_table"][b, key // page]), key % page


# prefix and own keys through the 16-row kernel; without a prefix; own keys alone there; the
# prefix as one stream pair and as several; own keys of many rows as tcgen05 jobs, 128 rows and more
EACH_KERNEL = [(2, 1, 8, 2, 64, 300, [5, 40], 16), (3, 2, 12, 2, 128, 0, [9, 2, 300], 32), (20, 1, 8, 2, 128, 700, [1 + 9 * i for i in range(20)], 64),
               (70, 2, 4, 2, 64, 1500, [2 + i for i in range(70)], 16), (2, 20, 8, 2, 128, 260, [20, 300], 16),
               (2, 70, 4, 1, 64, 129, [70, 333], 32)]


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,prefix,own_len,page", EACH_KERNEL)
def test_nan_query_row_is_nan(type_, B, T, Hq, Hkv, D, prefix, own_len, page):
    args = inputs(B, T, Hq, Hkv, D, prefix, own_len, page, type_, seed=31)
    args["q"][1, T - 1, 2, 7] = math.nan
    got = check_special(args, type_)
    assert bool(torch.isnan(got[1, T - 1, 2]).all()) and int(torch.isnan(got).sum()) == D


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,prefix,own_len,page", EACH_KERNEL)
def test_nan_key_that_is_used_gives_nan(type_, B, T, Hq, Hkv, D, prefix, own_len, page):
    """The first own key of request 1, all that its first rows have there."""
    args = inputs(B, T, Hq, Hkv, D, prefix, [T if b == 1 else n for b, n in enumerate(own_len)], page, type_, seed=32)
    args["k_cache"][(*own_place(args, 1, 0), 1 % Hkv)] = math.nan
    got = check_special(args, type_)
    assert int(torch.isnan(got).sum()) == T * (Hq // Hkv) * D


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,prefix,own_len,page", [c for c in EACH_KERNEL if c[1] > 1] + [
    (1, 5, 4, 2, 128, 0, [5], 16), (3, 3, 6, 2, 64, 40, [1, 2, 19], 32), (1, 200, 1, 1, 64, 0, [290], 64)])
def test_a_later_tokens_value_does_not_reach_earlier_rows(type_, value, B, T, Hq, Hkv, D, prefix, own_len, page):
    """Values of the last tokens of a request, which its earlier tokens do not see, are NaN or infinite."""
    args = inputs(B, T, Hq, Hkv, D, prefix, own_len, page, type_, seed=33)
    b, n = B - 1, own_len[B - 1]
    args["v_cache"][(*own_place(args, b, n - 1), 0, 3)] = value
    args["v_cache"][(*own_place(args, b, n - 2), Hkv - 1, D - 1)] = -value
    got = check_special(args, type_)
    assert bool(torch.isfinite(got[:, :T - 2]).all()) and bool(torch.isfinite(got[:b]).all())
    assert not bool(torch.isfinite(got[b, T - 1, 0, 3])) and not bool(torch.isfinite(got[b, T - 1, Hq - 1, D - 1]))


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,prefix,own_len,page", EACH_KERNEL)
def test_scores_that_are_all_minus_infinity(type_, B, T, Hq, Hkv, D, prefix, own_len, page):
    """0 / 0, not the zeros of a row without a key; beside finite scores they count for nothing."""
    args = inputs(B, T, Hq, Hkv, D, prefix, own_len, page, type_, seed=34)
    args["q"][..., 0] = 1.0
    for table, n in [(args["prefix_table"], prefix)] + [(args["own_table"][b], own_len[b]) for b in range(0, B, 2)]:
        for j in range(0, n, page):
            args["k_cache"][int(table[j // page]), :min(page, n - j), 0, 0] = -math.inf
    got = check_special(args, type_)
    G, last = Hq // Hkv, T - 1
    assert bool(torch.isnan(got[0, last, :G]).all()) and bool(torch.isfinite(got[1, last]).all())


def test_bounds_of_nearly_31_bits():
    """A table of 2^31 keys a request, of which a few are there, by a call of enough requests
    for one range each."""
    args = inputs(80, 1, 8, 8, 64, 20, [i % 7 for i in range(80)], 256, seed=12, own_pages=1)
    wide = torch.full((80, 1 << 23), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :1] = args["own_table"]
    for most in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 65):
        check({**args, "own_table": wide}, "f16", max_own=most)
