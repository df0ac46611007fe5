"""GPU tests of qmv_lora_add against its definition in 64 bits.

Tolerance, from the arithmetic: weights and fp16 activations are exact in every product;
what is held in pieces (fp32 activations, A x) keeps at least 21 bits, 2^-21 each; fp32
sums of at most 2^14 terms are taken over at most 64 dependent steps per chain (2^-23
each where a step truncates). Together below 2e-5 of the sum over absolute values, and
one rounding (2^-23) of base and of the output.
"""
import pytest
import torch

import decode_ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def inputs(M, N, K, R, L, x="f16", w="f16", seed=0, adapter=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if adapter is None:
        adapter = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    else:
        adapter = torch.tensor(adapter, dtype=torch.int32, device="cuda")
    return dict(x=r(M, K).to(TYPES[x]), a=(r(L, R, K) / max(K, 1) ** 0.5).to(TYPES[w]), b=r(L, N, R).to(TYPES[w]),
                adapter=adapter, scale=torch.rand((L,), generator=g, device="cuda") + 0.5, base=r(M, N))


def check(args, **kw):
    import gemm_qmv_quantize_gb300 as q
    y, bound = decode_ref.lora(**args)
    got = q.qmv_lora_add(**args, **kw)
    tol = 2e-5 * bound + 2.0 ** -22 * (args["base"].double().abs() + y.abs()) + 1e-30
    err = (got.double() - y).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    return got


@pytest.mark.parametrize("x,w", [("f16", "f16"), ("f16", "bf16"), ("f32", "f16"), ("f32", "bf16")])
@pytest.mark.parametrize("M,N,K,R,L", [
    (1, 1, 8, 8, 1), (1, 17, 40, 8, 3), (2, 130, 264, 16, 2), (5, 1000, 520, 24, 3), (7, 257, 1032, 40, 2),
    (9, 333, 4096, 64, 4), (33, 129, 512, 136, 5), (96, 260, 768, 32, 7), (3, 64, 2056, 256, 2), (8, 100, 17408, 16, 2)])
def test_sizes_and_types(M, N, K, R, L, x, w):
    check(inputs(M, N, K, R, L, x, w, seed=M * 1000 + N))


@pytest.mark.parametrize("adapter", [
    [0] * 40,                                             # all rows one adapter
    list(range(40)),                                      # each its own
    [-1] * 40,                                            # none at all
    [39, -1, 0, 0, 39, 40, 1000, -7] * 5,                 # shared, none, outside 0..L-1
    [1] * 17 + [0] * 9 + [-1] + [1] * 13])                # groups of odd sizes, apart
def test_who_shares_what(adapter):
    check(inputs(40, 300, 1024, 16, 40, "f16", "bf16", seed=3, adapter=adapter))


def test_in_place_and_rows_without_adapter():
    args = inputs(6, 500, 512, 16, 2, seed=5, adapter=[0, -1, 1, 0, 5, -1])
    y, bound = decode_ref.lora(**args)
    base = args["base"].clone()
    got = check(args, out=args["base"])
    assert got.data_ptr() == args["base"].data_ptr()
    for m in (1, 4, 5):
        assert torch.equal(got[m], base[m])


def test_large_fp32_activations_keep_their_range():
    args = inputs(3, 64, 256, 8, 2, "f32", "f16", seed=6)
    args["x"] *= 1e6                                       # beyond fp16's range
    check(args)


def test_no_adapters_and_empty_sum():
    import gemm_qmv_quantize_gb300 as q
    for args in (inputs(3, 50, 64, 8, 0, adapter=[0, 1, -1]), inputs(3, 50, 0, 8, 2)):
        assert torch.equal(q.qmv_lora_add(**args), args["base"])
    args = inputs(0, 50, 64, 8, 2)
    assert q.qmv_lora_add(**args).shape == (0, 50)


def test_same_call_same_bits_and_other_streams():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(20, 700, 2048, 32, 4, "f16", "bf16", seed=8)
    first = q.qmv_lora_add(**args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = q.qmv_lora_add(**args)
    third = torch.empty_like(first)
    q.qmv_lora_add(**args, out=third, stream=s)
    s.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)


def test_chained_calls_with_launch_overlap():
    """The output of one call is the next one's base, launches overlapping."""
    import gemm_qmv_quantize_gb300 as q
    args = inputs(4, 256, 256, 8, 3, seed=9)
    plain = args["base"]
    for _ in range(6):
        plain = q.qmv_lora_add(**{**args, "base": plain})
    try:
        q.set_launch_overlap(True)
        y = args["base"]
        for _ in range(6):
            y = q.qmv_lora_add(**{**args, "base": y})
        torch.cuda.synchronize()
    finally:
        q.set_launch_overlap(False)
    assert torch.equal(y, plain)


def test_refusals():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(2, 32, 64, 8, 2)
    with pytest.raises(TypeError):
        q.qmv_lora_add(**{**args, "x": args["x"].bfloat16()})
    with pytest.raises(TypeError):
        q.qmv_lora_add(**{**args, "b": args["b"].bfloat16()})
    with pytest.raises(ValueError):
        q.qmv_lora_add(**{**args, "b": args["b"][:, :-1].contiguous()})
    with pytest.raises(ValueError):
        q.qmv_lora_add(**{**args, "a": args["a"].transpose(1, 2).contiguous().transpose(1, 2)})
    with pytest.raises(ValueError):
        q.qmv_lora_add(**args, workspace=torch.empty((4,), dtype=torch.uint8, device="cuda"))
    with pytest.raises(q.QmvError):
        q.qmv_lora_add(**inputs(2, 32, 64, 12, 2))         # rank not a multiple of 8
    with pytest.raises(q.QmvError):
        q.qmv_lora_add(**inputs(97, 32, 64, 8, 2))         # more rows than a projection takes


def test_one_workspace_for_a_shrinking_batch():
    import gemm_qmv_quantize_gb300 as q
    ws = torch.empty((q.qmv_lora_add_workspace(96, 64, 4096),), dtype=torch.uint8, device="cuda")
    for M in (96, 75, 20, 1):
        check(inputs(M, 130, 4096, 64, 5, seed=M), workspace=ws)


@pytest.mark.parametrize("w", ["f16", "bf16"])
@pytest.mark.parametrize("x", ["f32", "f16"])
def test_infinite_activations(x, w):
    import gemm_qmv_quantize_gb300 as q
    args = inputs(3, 200, 256, 16, 2, x, w, seed=10, adapter=[0, 1, 0])
    args["a"], args["b"] = (t.abs().clamp(min=1e-3) for t in (args["a"], args["b"]))   # no 0 x inf, no inf - inf
    args["x"][1, 5] = -float("inf")
    y, _ = decode_ref.lora(**args)
    got = q.qmv_lora_add(**args).double()
    assert bool(torch.isneginf(got[1]).all()) and bool(torch.isneginf(y[1]).all())
    assert bool(torch.isfinite(got[::2]).all())


def test_products_beyond_fp32_and_infinite_weights():
    import gemm_qmv_quantize_gb300 as q
    args = inputs(3, 64, 256, 16, 2, "f32", "f16", seed=11, adapter=[0, 1, 0])
    args["x"], args["b"] = torch.zeros_like(args["x"]), args["b"].abs().clamp(min=1e-3)
    args["x"][0, 0], args["x"][1, 0] = 3e38, 2.0
    args["a"][:, :, 0] = 60000.0
    args["b"][1, 7, 3] = float("inf")
    got = q.qmv_lora_add(**args)
    assert bool(torch.isposinf(got[0]).all())              # A x is past fp32's range
    assert bool(torch.isposinf(got[1, 7])) and int(torch.isfinite(got[1]).sum()) == 63
    assert torch.equal(got[2], args["base"][2])


def test_sums_longer_than_a_grid_has_ranges():
    import gemm_qmv_quantize_gb300 as q
    K = (1 << 28) + (1 << 15)
    x = torch.zeros((1, K), dtype=torch.float16, device="cuda")
    x[0, ::1 << 20] = 1.0
    x[0, -1] = 1.0
    one = lambda *s, dtype=torch.float16: torch.ones(s, dtype=dtype, device="cuda")  # noqa: E731
    y = q.qmv_lora_add(x, one(1, 8, K), one(1, 5, 8), torch.zeros((1,), dtype=torch.int32, device="cuda"),
                       one(1, dtype=torch.float32), torch.zeros((1, 5), device="cuda"))
    assert y.tolist() == [[8.0 * 258] * 5]


@pytest.mark.parametrize("R", [128, 136, 256])
def test_full_batch_of_high_ranks(R):
    """Grids of three and of two CTAs an SM."""
    check(inputs(96, 1500, 512, R, 96, "f16", "bf16", seed=R, adapter=[(7 * i) % 96 for i in range(96)]))


@pytest.mark.parametrize("bits", [0x7f800001, 0x7fc00000, -1])
def test_nan_of_any_payload_stays_nan(bits):
    import gemm_qmv_quantize_gb300 as q
    args = inputs(3, 50, 256, 8, 2, "f32", "f16", seed=12, adapter=[0, 1, 0])
    args["x"].view(torch.int32)[1, 9] = bits
    got = q.qmv_lora_add(**args)
    assert bool(torch.isnan(got[1]).all()) and bool(torch.isfinite(got[::2]).all())
