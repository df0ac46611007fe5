"""Argument validation of the operators over a cache of 8 bits, of the norms and of sampling,
without a GPU: refusals and empty calls answer before any CUDA call. Only pointer values are
passed, never followed. And the binding's refusals, on tensors that say they are on a device."""
import random

import pytest
import torch

from test_decode_abi_host import ALIGN, BF16, BIG, F16, F32, NULL, OK, P, SHAPE, call, lib  # noqa: F401
from test_decode_binding_host import device_zero, on  # noqa: F401

APPEND = dict(qkv=P, positions=P, table=P, axis_of_pair=bytes(64), slots=P, q_norm=P, k_norm=P, eps=1e-6, q=P, k=P, v=P, type=F16,
              interleaved=0, M=4, Hq=8, Hkv=2, D=128, rot=128, axes=1, n_positions=100, n_slots=64, stream=None)
APPEND8 = {}
for _name, _value in APPEND.items():
    APPEND8[_name] = _value
    if _name == "v":
        APPEND8.update(k_scale=P, v_scale=P)

BOTH = [
    (dict(type=F32), SHAPE), (dict(M=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=132), SHAPE), (dict(D=264), SHAPE),
    (dict(rot=136), SHAPE), (dict(rot=20), SHAPE), (dict(rot=-8), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE),
    (dict(n_positions=0), SHAPE), (dict(n_slots=-1), SHAPE), (dict(axis_of_pair=bytes([0] * 63 + [1])), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(qkv=0), NULL), (dict(positions=0), NULL), (dict(table=0), NULL), (dict(axis_of_pair=None), NULL), (dict(slots=0), NULL),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL),
    (dict(qkv=P + 4), ALIGN), (dict(table=P + 8), ALIGN), (dict(slots=P + 4), ALIGN), (dict(k=P + 2), ALIGN), (dict(q_norm=P + 4), ALIGN),
    (dict(k_norm=P + 8), ALIGN), (dict(M=0, qkv=0), OK)]


@pytest.mark.parametrize("changes,status", BOTH + [(dict(Hkv=70000), SHAPE)])
def test_norm_rope_append(lib, changes, status):  # noqa: F811
    assert call(lib.qmv_norm_rope_append, APPEND, **changes) == status


@pytest.mark.parametrize("changes,status", BOTH + [
    (dict(D=96), SHAPE), (dict(D=256, rot=64), SHAPE), (dict(n_slots=40), SHAPE), (dict(k_scale=0), NULL), (dict(v_scale=0), NULL),
    (dict(k_scale=P + 2), ALIGN)])
def test_rope_append_e4m3(lib, changes, status):  # noqa: F811
    assert call(lib.qmv_rope_append_e4m3, APPEND8, **changes) == status


ATTENTION = dict(q=P, k=P, v=P, ks=P, vs=P, type=BF16, n_pages=100, page=16, table=P, table_pages=40, lens=P, max_len=600, scale=0.1,
                 out=P, workspace=P, ws_bytes=BIG, B=3, T=2, Hq=8, Hkv=2, D=128, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(type=F32), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(T=0), SHAPE), (dict(Hq=7), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(D=96), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE), (dict(max_len=641), SHAPE),
    (dict(max_len=-1), SHAPE), (dict(max_len=(1 << 30) + 1, table_pages=1 << 27), SHAPE), (dict(n_pages=0), SHAPE), (dict(n_pages=-1), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(ws_bytes=100), SHAPE),
    (dict(T=1 << 20), SHAPE), (dict(B=65535, T=1 << 15), SHAPE),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(ks=0), NULL), (dict(vs=0), NULL), (dict(table=0), NULL),
    (dict(lens=0), NULL), (dict(out=0), NULL), (dict(workspace=0), NULL),
    (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(out=P + 8), ALIGN), (dict(lens=P + 2), ALIGN), (dict(ks=P + 1), ALIGN),
    (dict(workspace=P + 8), ALIGN), (dict(B=0, q=0, out=0), OK)])
def test_paged_attention_e4m3(lib, changes, status):  # noqa: F811
    assert call(lib.qmv_paged_attention_e4m3, ATTENTION, **changes) == status


def test_paged_attention_e4m3_workspace(lib):  # noqa: F811
    need = lib.qmv_paged_attention_e4m3_workspace
    for bad in ((-1, 2, 8, 2, 128, 500), (3, 0, 8, 2, 128, 500), (3, 2, 8, 3, 128, 500), (3, 2, 8, 2, 100, 500), (3, 2, 8, 2, 128, -1)):
        assert need(*bad) == SHAPE
    rng = random.Random(3)
    for _ in range(5000):      # that of the largest serves all
        Hkv = rng.choice([1, 2, 4, 8, 16])
        heads = (Hkv * rng.randint(1, 10), Hkv, rng.choice([64, 128]))
        B, T, n = int(4000 ** rng.random()), rng.choice([1, 1, 2, 5, 8, 30, 96]), int(10 ** 6 * rng.random())
        most = need(B, T, *heads, n)
        assert most > 0
        assert most >= need(rng.randint(0, B), rng.randint(1, T), *heads, rng.randint(0, n))


SAMPLE = dict(logits=P, u=P, temperature=P, top_k=P, top_p=P, min_p=P, token=P, prob=P, M=3, V=1000, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(M=-1), SHAPE), (dict(M=65536), SHAPE), (dict(V=0), SHAPE), (dict(V=-5), SHAPE), (dict(V=524289), SHAPE),
    (dict(logits=0), NULL), (dict(u=0), NULL), (dict(token=0), NULL), (dict(logits=P + 2), ALIGN), (dict(top_k=P + 1), ALIGN),
    (dict(prob=P + 2), ALIGN), (dict(M=0, logits=0, token=0), OK)])
def test_sample(lib, changes, status):  # noqa: F811
    assert call(lib.qmv_sample, SAMPLE, **changes) == status


def tensors(op, device):
    half, i32, e4m3 = torch.float16, torch.int32, torch.float8_e4m3fn
    new = lambda *s, dtype=torch.float32: on(device, *s, dtype=dtype)  # noqa: E731
    cache, rope = (4, 16, 2, 64), dict(qkv=new(3, 6 * 64), positions=new(1, 3, dtype=i32), table=new(9, 32, 2), axis_of_pair=bytes(32),
                                       slots=new(3, dtype=torch.int64), q_norm=new(64), k_norm=new(64), out=new(3, 2, 64, dtype=half))
    codes = dict(k_cache=new(*cache, dtype=e4m3), v_cache=new(*cache, dtype=e4m3), k_scale=new(4, 1, 2), v_scale=new(4, 1, 2))
    return {
        "qmv_norm_rope_append": lambda: dict(rope, k_cache=new(*cache, dtype=half), v_cache=new(*cache, dtype=half)),
        "qmv_rope_append_e4m3": lambda: dict(rope, **codes),
        "qmv_paged_attention_e4m3": lambda: dict(codes, q=new(2, 1, 4, 64, dtype=half), table=new(2, 1, dtype=i32), lens=new(2, dtype=i32),
                                                 out=new(2, 1, 4, 64, dtype=half), workspace=new(1 << 20, dtype=torch.uint8)),
        "qmv_sample": lambda: dict(logits=new(2, 100), u=new(2), temperature=new(2), top_k=new(2, dtype=i32), top_p=new(2), min_p=new(2),
                                   out=new(2, dtype=i32), prob=new(2)),
    }[op]()


OPERATORS = ["qmv_norm_rope_append", "qmv_rope_append_e4m3", "qmv_paged_attention_e4m3", "qmv_sample"]


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_on_different_devices(op, device_zero):  # noqa: F811
    import gemm_qmv_quantize_gb300 as q
    for name, t in tensors(op, 1).items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError, match="cuda:1"):
                getattr(q, op)(**{**tensors(op, 0), name: t})


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_that_are_not_on_the_current_device(op, device_zero):  # noqa: F811
    import gemm_qmv_quantize_gb300 as q
    with pytest.raises(ValueError, match="current device is cuda:0"):
        getattr(q, op)(**tensors(op, 1))


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_on_the_cpu(op, device_zero):  # noqa: F811
    import gemm_qmv_quantize_gb300 as q
    for name, t in tensors(op, 0).items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError, match="must be a CUDA tensor"):
                getattr(q, op)(**{**tensors(op, 0), name: torch.zeros(t.shape, dtype=t.dtype)})


def test_the_example_step_refuses():
    from gemm_qmv_quantize_gb300.decode_step import DecodeStep
    with pytest.raises(ValueError, match="f16 or e4m3"):
        DecodeStep(1, 16, 4, cache="int8")
    with pytest.raises(ValueError, match="do not end with a page"):
        DecodeStep(1, 17, 4, page=16, cache="e4m3")
