"""GPU tests of qmv_sample against its definition in 64 bits.

Tolerance: a weight is within 2^-32 of its value and 2^-44 of the largest, so a sum of them is
within 2^-31 of its value and 2^-44 a token: the token is the one that u falls to, or its
neighbour where u is nearer than that to the border between them; the probability, rounded to
fp32, is within 2^-23 of its value.
"""
import math

import pytest
import torch

import cache8_ref

pytestmark = pytest.mark.gpu


def inputs(M, V, spread=3.0, top_k=None, top_p=None, min_p=None, temperature=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = lambda v, dtype: None if v is None else torch.full((M,), v, dtype=dtype, device="cuda")  # noqa: E731
    return dict(logits=torch.randn((M, V), generator=g, device="cuda") * spread, u=torch.rand((M,), generator=g, device="cuda"),
                temperature=torch.rand((M,), generator=g, device="cuda") + 0.3 if temperature else None,
                top_k=full(top_k, torch.int32), top_p=full(top_p, torch.float32), min_p=full(min_p, torch.float32))


def run(args, **kw):
    import gemm_qmv_quantize_gb300 as q
    prob = torch.empty((args["logits"].shape[0],), device="cuda")
    return q.qmv_sample(**args, prob=prob, **kw), prob


def check(args):
    token, prob = run(args)
    V = args["logits"].shape[1]
    of = lambda name, m, none: none if args[name] is None else args[name][m].item()  # noqa: E731
    for m in range(len(token)):
        got = int(token[m])
        wrong = []
        # A top-p's border is p S, and both S and the sum before a token are within e = 2^-31 + 2^-44 V of S (which is
        # 1 at least) of their values: they compare as at some p' with |p' - p| <= e (1 + p). So a token that is on the border but
        # for that is kept or not; equal heavy tokens, whose sums meet p S exactly but for tokens of 2^-49, are.
        p = of("top_p", m, 1.0)
        e = (2.0 ** -31 + 2.0 ** -44 * V) * (1 + p)
        for top_p in (p, p - e, p + e) if 0 < p < 1 else (p,):
            ids, w = cache8_ref.kept(args["logits"][m], of("temperature", m, 1.0), of("top_k", m, 0), top_p, of("min_p", m, 0.0))
            wrong.append(not_drawn(ids, w, got, float(prob[m]), float(args["u"][m])))
            if wrong[-1] is None:
                break
        assert wrong[-1] is None, (m, got, wrong)
    return token


def not_drawn(ids, w, got, prob, u):
    """Why the token is not the one that u falls to among the tokens ids of weights w, or None."""
    if len(ids) == 0:
        return None if got == -1 and prob == 0 else "no token is kept"
    at = (ids == got).nonzero()
    if at.numel() != 1:
        return f"not among the {len(ids)} kept"
    at = int(at)
    upto = torch.cumsum(w, 0)
    total = float(upto[-1])
    target = min(max(u, 0.0), 1 - 2.0 ** -24) * total
    near = 2.0 ** -31 * total + 2.0 ** -44 * len(ids)
    if not float(upto[at] - w[at]) - near <= target < float(upto[at]) + near:
        return f"{target} is not in {float(upto[at] - w[at])} .. {float(upto[at])}"
    if not abs(prob - float(w[at]) / total) <= 2.0 ** -23 * float(w[at]) / total + 2.0 ** -40:
        return f"probability {prob}, not {float(w[at]) / total}"
    return None


@pytest.mark.parametrize("filters", [{}, dict(top_k=5), dict(top_p=0.8), dict(min_p=0.1), dict(top_k=50, top_p=0.95),
                                     dict(top_k=200, top_p=0.5, min_p=0.02)])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (2, 31), (5, 1000), (4, 4097), (2, 32000), (3, 50257), (2, 151936)])
def test_sizes_and_filters(M, V, filters):
    check(inputs(M, V, seed=M + V, **filters))


@pytest.mark.parametrize("spread", [0.0, 0.01, 0.3, 1.0, 10.0, 100.0])
@pytest.mark.parametrize("filters", [dict(top_k=777), dict(top_p=0.3), dict(top_k=3000, top_p=0.999)])
def test_flat_and_steep(spread, filters):
    check(inputs(3, 20011, spread, seed=int(spread * 100), **filters))


@pytest.mark.parametrize("spread", [0.0, 0.001, 0.02])
def test_a_small_top_k_among_many_alike(spread):
    """The bin with the cut holds more tokens than are ranked at once."""
    check(inputs(4, 20011, spread, top_k=100, top_p=0.9, seed=11))
    check(inputs(4, 20011, spread, top_k=100, min_p=0.5, seed=12))


@pytest.mark.parametrize("filters", [dict(top_k=50), dict(top_k=50, top_p=0.95), dict(top_k=5000, top_p=0.9), dict(top_p=0.999999), {}])
def test_fewer_tokens_of_any_weight_than_top_k(filters):
    check(inputs(6, 30000, 60.0, seed=13, **filters))


@pytest.mark.parametrize("V", [7, 300, 9000])
def test_ties_go_to_the_lowest_index(V):
    """Logits of few distinct values: cuts fall among equals. Sums of equal weights are exact here."""
    g = torch.Generator(device="cuda").manual_seed(V)
    for k, p in ((3, 1.0), (V // 2 + 1, 1.0), (0, 0.5), (V // 3 + 1, 0.25)):
        args = inputs(4, V, seed=V, top_k=k, top_p=p, temperature=False)
        args["logits"] = torch.randint(0, 3, (4, V), generator=g, device="cuda").float()
        args["logits"][0] = 1.5
        args["logits"][1] = torch.where(torch.arange(V, device="cuda") % 2 == 0, -0.0, 0.0)
        check(args)


def test_an_exact_share_of_equal_tokens():
    args = inputs(3, 8, top_p=0.5, temperature=False)
    args["logits"].fill_(2.0)                                  # 0.5 of eight equals: the first four
    args["u"] = torch.tensor([0.0, 0.74999, 0.99999], device="cuda")
    assert run(args)[0].tolist() == [0, 2, 3]


def test_where_the_random_number_falls():
    args = inputs(6, 4, temperature=False)
    args["logits"][:] = torch.log(torch.tensor([1.0, 2.0, 4.0, 1.0], device="cuda"))
    args["u"] = torch.tensor([0.0, 0.124, 0.126, 0.374, 0.376, 0.876], device="cuda")
    assert run(args)[0].tolist() == [0, 0, 1, 1, 2, 3]
    args["u"] = torch.tensor([-1.0, math.nan, 1.0, 7.0, math.inf, -math.inf], device="cuda")
    assert run(args)[0].tolist() == [0, 0, 3, 3, 3, 0]


def test_greedy_rows():
    args = inputs(6, 5000, top_k=40, top_p=0.9, seed=1)
    args["temperature"][:] = torch.tensor([0.0, -1.0, math.nan, -math.inf, 1e-30, 1e-45], device="cuda")
    token, prob = run(args)
    assert torch.equal(token.long(), args["logits"].argmax(1)) and bool((prob == 1).all())
    args["logits"][:, [7, 4000]] = 50.0
    assert run(args)[0][:4].tolist() == [7] * 4


def test_settings_that_keep_one_token_or_all():
    args = inputs(4, 3000, seed=2)
    best = args["logits"].argmax(1)
    for one in (dict(top_k=1), dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=1.5), dict(top_p=1e-30), dict(top_p=1e-45)):
        assert torch.equal(run(inputs(4, 3000, seed=2, **one))[0].long(), best), one
    plain = run(args)
    for all_ in (dict(top_k=0), dict(top_k=-3), dict(top_k=3000), dict(top_k=10 ** 9), dict(top_p=1.0), dict(top_p=2.0),
                 dict(top_p=math.nan), dict(min_p=0.0), dict(min_p=-1.0), dict(min_p=math.nan)):
        got = run(inputs(4, 3000, seed=2, **all_))
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1]), all_


def test_each_row_has_its_own_settings():
    args = inputs(8, 10007, top_k=0, top_p=1.0, min_p=0.0, seed=3)
    args["temperature"] = torch.tensor([0.0, 0.5, 1.0, 2.0, 1.0, 0.7, 100.0, math.inf], device="cuda")
    args["top_k"] = torch.tensor([0, 3, 0, 500, 1, 10007, 10006, 2000], dtype=torch.int32, device="cuda")
    args["top_p"] = torch.tensor([1.0, 0.9, 0.9, 0.99, 0.5, 0.999, 0.3, 0.6], device="cuda")
    args["min_p"] = torch.tensor([0.0, 0.0, 0.2, 0.001, 0.5, 0.0, 0.9, 0.0], device="cuda")
    check(args)


def test_special_logits():
    args = inputs(7, 999, top_k=20, top_p=0.9, seed=4)
    x = args["logits"]
    x[0].fill_(-math.inf)
    x[1].fill_(math.nan)
    x[2] = -math.inf
    x[2, 500] = -3e38
    x[3, [5, 600]] = math.inf
    x[4, ::2] = math.nan
    x[5] = torch.finfo(torch.float32).min
    x[6, 3], x[6, 4] = torch.finfo(torch.float32).max, -torch.finfo(torch.float32).max
    token = check(args)
    assert token[:3].tolist() == [-1, -1, 500] and int(token[3]) in (5, 600) and int(token[4]) % 2 == 1
    args = {**args, "top_k": None, "top_p": None}
    check(args)


def test_masked_logits_are_never_drawn():
    args = inputs(64, 1003, 0.5, seed=5)
    args["logits"][:, ::3] = -math.inf
    args["u"] = torch.linspace(0, 1, 64, device="cuda")
    assert bool((run(args)[0] % 3 != 0).all())


def test_frequencies_follow_the_probabilities():
    """Evenly spaced random numbers: each token's share of them is within one of its probability's."""
    M, V = 4096, 50
    args = inputs(M, V, 1.0, top_p=0.9, temperature=False, seed=6)
    args["logits"][:] = args["logits"][:1].clone()
    args["u"] = (torch.arange(M, device="cuda") + 0.5) / M
    ids, w = cache8_ref.kept(args["logits"][0], 1.0, 0, 0.8999999761581421, 0.0)
    count = torch.bincount(run(args)[0].long(), minlength=V)[ids]
    assert bool(((count - M * w / w.sum()).abs() <= 1.0).all()) and int(count.sum()) == M


def test_rows_that_start_anywhere():
    """Rows of odd length begin on every 4-byte boundary of 16 bytes, and so may the first."""
    whole = torch.randn((7 * 4099 + 4,), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda") * 3
    for skew in range(4):
        args = inputs(7, 4099, top_k=100, top_p=0.9, seed=8)
        args["logits"] = whole[skew:skew + 7 * 4099].view(7, 4099)
        check(args)


@pytest.mark.parametrize("V", [37, 8191, 70001])
@pytest.mark.parametrize("spread", [2.0, 4.0, 8.0, 30.0])
def test_a_top_p_alone_of_narrow_and_wide_rows(spread, V):
    for top_p in (0.2, 0.9, 0.99, 0.9999):
        check(inputs(3, V, spread, top_p=top_p, min_p=0.001 if spread == 8.0 else None, seed=int(spread) + V))


@pytest.mark.parametrize("top_p", [0.5, 0.95, 0.9999])
def test_wide_rows_whose_tokens_are_nearly_all_alike(top_p):
    """Some light tokens make the range wide, though all but those count; or a few heavy ones, and a cut far among the others."""
    args = inputs(4, 20011, 0.01, top_p=top_p, temperature=False, seed=14)
    x = args["logits"]
    x[:3, 5:20011:4000] = -60.0
    x[1, ::2], x[1, 1::7] = -math.inf, math.nan
    x[2] = torch.where(x[2] > -1, 0.0, x[2])
    x[2, 11::13] = -0.0
    x[3] = torch.where(torch.arange(20011, device="cuda") % 1000 == 17, 9.0, x[3] - 25.0)
    check(args)


@pytest.mark.parametrize("dense_first", [True, False])
def test_some_shares_with_lists_and_some_without(dense_first):
    """Ten heavy tokens, all that are kept; half of the others, 2000 on end, just heavy enough to be listed, more than lists hold."""
    V = 70001
    args = inputs(4, V, 0.02, top_p=0.99, temperature=False, seed=17)
    x = args["logits"]
    half = torch.arange(V, device="cuda") // 2000 % 2 == 0
    x += torch.where(half == dense_first, -13.3, -40.0)
    x[:, 5] = -60.0
    x[:, 3001:V:7000] = 0.0
    token = check(args)
    assert bool((token % 7000 == 3001).all())


def test_special_logits_of_wide_rows():
    args = inputs(5, 9001, 6.0, top_p=0.9, temperature=False, seed=15)
    x = args["logits"]
    x[0, ::3] = math.nan
    x[1, 1::2] = -math.inf
    x[2, [4, 8000]] = math.inf
    x[3, :8000] = -80.0
    x[4, 77] = torch.finfo(torch.float32).max
    check(args)


def test_threads_largest_logits_in_a_few_places():
    """As many large logits as top_k in the parts of few threads; all of them in one."""
    args = inputs(3, 50001, 0.1, top_k=60, top_p=0.97, seed=16)
    args["logits"][0, 4096:4196] += 9.0
    args["logits"][1, 48000:48300] += 5.0
    args["logits"][2, :4] += 20.0
    check(args)


def test_a_large_vocabulary():
    for V in (300001, 524288):
        check(inputs(2, V, 2.0, top_p=0.95, seed=V))


def test_the_same_bits_again_and_in_a_graph():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(9, 151936, 1.0, top_k=5000, top_p=0.9, min_p=0.001, seed=9)
    plain, prob = run(args)
    out, p = torch.empty_like(plain), torch.empty_like(prob)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qmv_sample(**args, out=out, prob=p)
    for _ in range(3):
        out.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain) and torch.equal(p, prob)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = q.qmv_sample(**args, stream=s)
    s.synchronize()
    assert torch.equal(other, plain)


def test_empty_and_refusals():
    import gemm_qmv_quantize_gb300 as q
    assert q.qmv_sample(torch.empty((0, 50), device="cuda"), torch.empty((0,), device="cuda")).shape == (0,)
    args = inputs(2, 100, top_k=3)
    for bad in (dict(u=args["u"][:1]), dict(temperature=torch.ones((2, 1), device="cuda")), dict(logits=args["logits"].T)):
        with pytest.raises(ValueError):
            run({**args, **bad})
    for bad in (dict(top_k=args["top_k"].long()), dict(logits=args["logits"].half()), dict(u=args["u"].double())):
        with pytest.raises(TypeError):
            run({**args, **bad})
    with pytest.raises(q.QmvError):
        q.qmv_sample(torch.empty((1, 524289), device="cuda"), torch.empty((1,), device="cuda"))
    with pytest.raises(q.QmvError):
        q.qmv_sample(torch.empty((1, 0), device="cuda"), torch.empty((1,), device="cuda"))
