"""Argument validation of the decode-step operators, without a GPU: refusals and empty
calls answer before any CUDA call. Only pointer values are passed, never followed."""
import ctypes
import random

import pytest


@pytest.fixture(scope="module")
def lib():
    from gemm_qmv_quantize_gb300 import build
    build.build()
    import gemm_qmv_quantize_gb300 as q
    return q.lib()


OK, NULL, SHAPE, ALIGN = 0, -1, -2, -3
P = 0x10000
F32, F16, BF16 = 0, 1, 2
BIG = 1 << 40


def call(fn, defaults, **changes):
    assert set(changes) <= set(defaults)
    return fn(*{**defaults, **changes}.values())


LORA = dict(x=P, x_type=F16, a=P, b=P, w_type=BF16, adapter=P, scale=P, base=P, y=P, workspace=P, ws_bytes=BIG, M=4, N=64,
            K=128, R=16, L=2, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(x_type=BF16), SHAPE), (dict(x_type=7), SHAPE), (dict(w_type=F32), SHAPE), (dict(M=97), SHAPE), (dict(M=-1), SHAPE),
    (dict(R=0), SHAPE), (dict(R=12), SHAPE), (dict(R=264), SHAPE), (dict(K=132), SHAPE), (dict(K=-8), SHAPE),
    (dict(N=-1), SHAPE), (dict(N=1 << 31), SHAPE), (dict(L=-1), SHAPE), (dict(ws_bytes=0), SHAPE),
    (dict(x=0), NULL), (dict(a=0), NULL), (dict(b=0), NULL), (dict(adapter=0), NULL), (dict(scale=0), NULL),
    (dict(base=0), NULL), (dict(y=0), NULL), (dict(workspace=0), NULL),
    (dict(x=P + 8), ALIGN), (dict(a=P + 2), ALIGN), (dict(b=P + 8), ALIGN), (dict(adapter=P + 2), ALIGN),
    (dict(y=P + 1), ALIGN), (dict(workspace=P + 4), ALIGN),
    (dict(M=0, x=0, y=0), OK), (dict(N=0, x=0, y=0), OK), (dict(L=0, a=0, b=0), OK), (dict(K=0), OK)])
def test_lora_add(lib, changes, status):
    assert call(lib.qmv_lora_add, LORA, **changes) == status


def test_lora_add_workspace(lib):
    assert lib.qmv_lora_add_workspace(4, 16, 128) > 0
    for bad in ((97, 16, 128), (4, 15, 128), (4, 16, 127), (-1, 16, 128)):
        assert lib.qmv_lora_add_workspace(*bad) == SHAPE


ROPE = dict(qkv=P, positions=P, table=P, axis_of_pair=bytes(64), slots=P, q=P, k=P, v=P, type=F16, interleaved=0, M=4,
            Hq=8, Hkv=2, D=128, rot=128, axes=1, n_positions=100, n_slots=64, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(type=F32), SHAPE), (dict(M=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=132), SHAPE),
    (dict(D=264), SHAPE), (dict(rot=136), SHAPE), (dict(rot=20), SHAPE), (dict(rot=-8), SHAPE), (dict(axes=0), SHAPE),
    (dict(axes=5), SHAPE), (dict(n_positions=0), SHAPE), (dict(n_slots=-1), SHAPE),
    (dict(axis_of_pair=bytes([0] * 63 + [1])), SHAPE),
    (dict(qkv=0), NULL), (dict(positions=0), NULL), (dict(table=0), NULL), (dict(axis_of_pair=None), NULL),
    (dict(slots=0), NULL), (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL),
    (dict(qkv=P + 4), ALIGN), (dict(table=P + 8), ALIGN), (dict(slots=P + 4), ALIGN), (dict(k=P + 2), ALIGN),
    (dict(M=0, qkv=0), OK)])
def test_rope_append(lib, changes, status):
    assert call(lib.qmv_rope_append, ROPE, **changes) == status


ATTENTION = dict(q=P, k=P, v=P, type=BF16, n_pages=100, page=16, prefix_table=P, prefix_len=500, own_table=P, own_pages=4,
                 own_len=P, max_own=64, scale=0.1, out=P, workspace=P, ws_bytes=BIG, B=3, T=2, Hq=8, Hkv=2, D=128,
                 stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(type=F32), SHAPE), (dict(B=-1), SHAPE), (dict(T=0), SHAPE), (dict(Hq=7), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(D=96), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE),
    (dict(prefix_len=-1), SHAPE), (dict(max_own=65), SHAPE), (dict(max_own=-1), SHAPE), (dict(n_pages=0), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(prefix_table=0), NULL), (dict(own_table=0), NULL),
    (dict(own_len=0), NULL), (dict(out=0), NULL),
    (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(out=P + 8), ALIGN), (dict(own_len=P + 2), ALIGN),
    (dict(workspace=P + 8), ALIGN), (dict(B=0, q=0, out=0), OK)])
def test_prefix_attention(lib, changes, status):
    assert call(lib.qmv_prefix_attention, ATTENTION, **changes) == status


def test_prefix_attention_workspace(lib):
    assert lib.qmv_prefix_attention_workspace(3, 2, 8, 2, 128, 500, 64) >= 0
    for bad in ((-1, 2, 8, 2, 128, 500, 64), (3, 0, 8, 2, 128, 500, 64), (3, 2, 8, 3, 128, 500, 64),
                (3, 2, 8, 2, 100, 500, 64), (3, 2, 8, 2, 128, -1, 64), (3, 2, 8, 2, 128, 500, 1 << 31)):
        assert lib.qmv_prefix_attention_workspace(*bad) == SHAPE


LOGITS = dict(logits=P, tokens=P, max_history=100, prompt_len=P, total_len=P, repetition=P, presence=P, frequency=P,
              bias_tokens=P, bias_values=P, max_bias=4, mask=P, mask_row=P, n_masks=2, y=P, M=3, V=1000, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(M=-1), SHAPE), (dict(M=65536), SHAPE), (dict(V=-1), SHAPE), (dict(max_history=-1), SHAPE),
    (dict(max_bias=-1), SHAPE), (dict(n_masks=-1), SHAPE), (dict(mask_row=0), SHAPE),
    (dict(logits=0), NULL), (dict(y=0), NULL), (dict(tokens=0), NULL), (dict(prompt_len=0), NULL),
    (dict(total_len=0), NULL), (dict(bias_tokens=0), NULL), (dict(bias_values=0), NULL), (dict(mask=0), NULL),
    (dict(logits=P + 2), ALIGN), (dict(tokens=P + 1), ALIGN), (dict(mask=P + 2), ALIGN), (dict(frequency=P + 2), ALIGN),
    (dict(M=0, logits=0, y=0), OK), (dict(V=0, logits=0, y=0), OK)])
def test_penalize_logits(lib, changes, status):
    assert call(lib.qmv_penalize_logits, LOGITS, **changes) == status


def test_workspaces_are_64_bit(lib):
    assert lib.qmv_lora_add_workspace.restype is ctypes.c_int64
    assert lib.qmv_prefix_attention_workspace.restype is ctypes.c_int64


def test_lora_add_workspace_of_the_largest_serves_all(lib):
    need = lib.qmv_lora_add_workspace
    assert need(96, 64, 4096) >= need(75, 64, 4096) and need(96, 16, 16384) >= need(96, 16, 12288)
    rng = random.Random(1)
    for _ in range(5000):
        M, R, K = rng.randint(1, 96), 8 * rng.randint(1, 32), 8 * rng.randint(1, 3000)
        most = need(M, R, K)
        assert most >= need(rng.randint(0, M), R, K) and most >= need(M, 8 * rng.randint(1, R // 8), K)
        assert most >= need(M, R, 8 * rng.randint(0, K // 8))


def test_prefix_attention_workspace_of_the_largest_serves_all(lib):
    need = lib.qmv_prefix_attention_workspace
    assert need(64, 1, 40, 8, 128, 65536, 1024) >= need(45, 1, 40, 8, 128, 65536, 1024)
    rng = random.Random(2)
    any_of = lambda n: int(n ** rng.random())  # noqa: E731
    for _ in range(20000):
        Hkv = rng.choice([1, 2, 4, 8, 16])
        heads = (Hkv * rng.randint(1, 10), Hkv, rng.choice([64, 128]))
        B, T, prefix, own = any_of(400), rng.choice([1, 1, 2, 5, 8, 30, 96, 700]), any_of(200000) - 1, any_of(60000) - 1
        most = need(B, T, *heads, prefix, own)
        if most < 0:      # more rows than a call takes
            continue
        b, t, p, o = rng.randint(0, B), rng.randint(1, T), rng.randint(0, prefix), rng.randint(0, own)
        for fewer in ((b, T, prefix, own), (B, t, prefix, own), (B, T, p, own), (B, T, prefix, o), (b, t, p, o)):
            assert most >= need(fewer[0], fewer[1], *heads, *fewer[2:])
