"""Binding of the operators beside the matmuls in a batched decode step (include/qmv.h):
low-rank adapters, rotary positions (with norms of q and k) and the append to a paged cache
of 16 or 8 bits, attention over a shared prefix or over a cache of 8 bits, penalties, biases
and masks on logits, and sampling.

As in ``_binding``: tensors are checked for type, shape, contiguity and device, pointers and
sizes go to the C entry point of the same name, and all arithmetic runs in the library.
An output or a workspace that is not given is allocated for the call, from the memory of
its stream; a program that repeats calls keeps a workspace of the bytes that the
``_workspace`` function names for its largest batch.
"""
from __future__ import annotations

import functools
import math

import torch

from ._binding import QMV_OK, QmvError, _check, _need, _stream, lib

_F32, _F16, _BF16, _I32 = torch.float32, torch.float16, torch.bfloat16, torch.int32
_TYPE = {_F32: 0, _F16: 1, _BF16: 2}   # QMV_F32, QMV_F16, QMV_BF16
_16BIT = (_F16, _BF16)
_E4M3 = torch.float8_e4m3fn
_current_device = torch._C._cuda_getDevice


@functools.cache
def _fn(name: str):
    """The library's function (looked up once: a decode step's calls take microseconds)."""
    return getattr(lib(), name)


def _type(t: torch.Tensor, name: str, allowed) -> int:
    if t.dtype not in allowed:
        raise TypeError(f"{name}: expected {' or '.join(map(str, allowed))}, got {t.dtype}")
    return _TYPE[t.dtype]


def _is(t, name: str, dtype, shape, device: int):
    """_need, with the checks that pass in a few tenths of a microsecond first; and t is on
    the device of the call's other tensors (by number)."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()):
        _need(t, name, dtype, shape)
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's first tensor on cuda:{device}")


def _held(t, name: str, dtype, device: int):
    """_is for a tensor whose own shape the call goes by."""
    if not (t.dtype is dtype and t.get_device() == device and t.is_contiguous()):
        _need(t, name, dtype)
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's first tensor on cuda:{device}")


def _first(t, name: str, dtype) -> int:
    """_held for a call's first tensor: its device, which is the current one, where the
    library launches."""
    if not (t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        _need(t, name, dtype)
    device = t.get_device()
    if device != _current_device():
        raise ValueError(f"{name} is on cuda:{device}, the current device is cuda:{_current_device()}")
    return device


def _on(stream, device: int) -> int:
    """The handle of `stream`, or of the device's current one (without a Stream object for it,
    which costs as much as a launch)."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on `stream`, from the memory of that stream: a block that the
    current one has freed may still be in use by its queued work, which `stream` does not
    wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(buffer, need, device: int, stream):
    """`buffer`, or a new one of need() bytes for a call on `stream`."""
    if buffer is None:
        return _empty((need(),), torch.uint8, torch.device("cuda", device), stream)
    _held(buffer, "workspace", torch.uint8, device)
    return buffer


def _check_with(fn: str, status: int, buffer, need):
    """_check, naming a workspace that is too small."""
    if status != QMV_OK:
        if buffer.numel() < need():
            raise ValueError(f"workspace: {buffer.numel()} bytes, {fn} needs {need()}")
        _check(fn, status)


def _bytes(fn: str, n: int) -> int:
    if n < 0:
        raise QmvError(fn, n)
    return n


def qmv_lora_add_workspace(M: int, R: int, K: int) -> int:
    """Bytes of workspace of qmv_lora_add on M rows of K with adapters of rank R."""
    return _bytes("qmv_lora_add_workspace", _fn("qmv_lora_add_workspace")(M, R, K))


def qmv_lora_add(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapter: torch.Tensor, scale: torch.Tensor,
                 base: torch.Tensor, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """base fp32 [M, N] + scale[l] (x[m] A[l]^T) B[l]^T with l = adapter[m] (none where it
    is outside 0..L-1): x fp32 or fp16 [M, K], a [L, R, K] and b [L, N, R] fp16 or bf16,
    adapter int32 [M], scale fp32 [L]. out may be base."""
    M, K = x.shape
    L, R, _ = a.shape
    N = base.shape[1]
    xt, wt = _type(x, "x", (_F32, _F16)), _type(a, "a", _16BIT)
    dev = _first(x, "x", x.dtype)
    _is(a, "a", a.dtype, (L, R, K), dev)
    _is(b, "b", a.dtype, (L, N, R), dev)
    _is(adapter, "adapter", _I32, (M,), dev)
    _is(scale, "scale", _F32, (L,), dev)
    _is(base, "base", _F32, (M, N), dev)
    if out is None:
        out = _empty((M, N), _F32, base.device, stream)
    else:
        _is(out, "out", _F32, (M, N), dev)
    need = lambda: qmv_lora_add_workspace(M, R, K)  # noqa: E731
    ws = _workspace(workspace, need, dev, stream)
    status = _fn("qmv_lora_add")(
        x.data_ptr(), xt, a.data_ptr(), b.data_ptr(), wt, adapter.data_ptr(), scale.data_ptr(), base.data_ptr(),
        out.data_ptr(), ws.data_ptr(), ws.numel(), M, N, K, R, L, _on(stream, dev))
    if status != QMV_OK:
        _check_with("qmv_lora_add", status, ws, need)
    return out


def qmv_rope_table(n_positions: int, rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """fp32 [n_positions, rot/2, 2]: (cos, sin) of position * base^(-2i/rot), computed in
    64 bits and rounded once."""
    pairs = rot // 2
    inv = base ** -(torch.arange(pairs, dtype=torch.float64, device=device) / max(pairs, 1))
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32).contiguous()


def qmv_rope_append(qkv: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, axis_of_pair, slots: torch.Tensor,
                    k_cache: torch.Tensor, v_cache: torch.Tensor, interleaved: bool = False,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Turns q and k of qkv fp32 [M, (Hq + 2 Hkv) D] by their positions, int32 [axes, M],
    and writes k and v to slots int64 [M] of k_cache and v_cache [pages, page, Hkv, D]
    (negative slots are skipped); returns q [M, Hq, D] in the caches' type. table: fp32
    [n_positions, rot/2, 2] as of qmv_rope_table; axis_of_pair: rot/2 numbers (bytes, or a
    sequence), the axis of each pair. interleaved: pairs (2i, 2i+1), not (i, i + rot/2)."""
    pages, page, Hkv, D = k_cache.shape
    M, width = qkv.shape
    axes = positions.shape[0]
    n_positions, pairs, _ = table.shape
    heads, odd = divmod(width, D)
    if odd or heads <= 2 * Hkv:
        raise ValueError(f"qkv: rows of {width} are not q heads and 2 x {Hkv} heads of {D}")
    Hq = heads - 2 * Hkv
    if not isinstance(axis_of_pair, bytes):
        axis_of_pair = bytes(axis_of_pair)
    if len(axis_of_pair) != pairs:
        raise ValueError(f"axis_of_pair: expected {pairs} entries, got {len(axis_of_pair)}")
    dtype = k_cache.dtype
    t = _type(k_cache, "k_cache", _16BIT)
    dev = _first(qkv, "qkv", _F32)
    _is(positions, "positions", _I32, (axes, M), dev)
    _is(table, "table", _F32, (n_positions, pairs, 2), dev)
    _is(slots, "slots", torch.int64, (M,), dev)
    _held(k_cache, "k_cache", dtype, dev)
    _is(v_cache, "v_cache", dtype, k_cache.shape, dev)
    if out is None:
        out = _empty((M, Hq, D), dtype, qkv.device, stream)
    else:
        _is(out, "out", dtype, (M, Hq, D), dev)
    status = _fn("qmv_rope_append")(
        qkv.data_ptr(), positions.data_ptr(), table.data_ptr(), axis_of_pair, slots.data_ptr(), out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), t, 1 if interleaved else 0, M, Hq, Hkv, D, 2 * pairs, axes,
        n_positions, pages * page, _on(stream, dev))
    if status != QMV_OK:
        _check("qmv_rope_append", status)
    return out


def _rope_args(qkv, positions, table, axis_of_pair, slots, k_cache, v_cache, q_norm, k_norm, cache_type):
    """What both appends with norms check and pass on: (device, Hq, axis_of_pair)."""
    pages, page, Hkv, D = k_cache.shape
    M, width = qkv.shape
    n_positions, pairs, _ = table.shape
    heads, odd = divmod(width, D)
    if odd or heads <= 2 * Hkv:
        raise ValueError(f"qkv: rows of {width} are not q heads and 2 x {Hkv} heads of {D}")
    if not isinstance(axis_of_pair, bytes):
        axis_of_pair = bytes(axis_of_pair)
    if len(axis_of_pair) != pairs:
        raise ValueError(f"axis_of_pair: expected {pairs} entries, got {len(axis_of_pair)}")
    dev = _first(qkv, "qkv", _F32)
    _is(positions, "positions", _I32, (positions.shape[0], M), dev)
    _is(table, "table", _F32, (n_positions, pairs, 2), dev)
    _is(slots, "slots", torch.int64, (M,), dev)
    _held(k_cache, "k_cache", cache_type, dev)
    _is(v_cache, "v_cache", cache_type, k_cache.shape, dev)
    if q_norm is not None:
        _is(q_norm, "q_norm", _F32, (D,), dev)
    if k_norm is not None:
        _is(k_norm, "k_norm", _F32, (D,), dev)
    return dev, heads - 2 * Hkv, axis_of_pair


def _ptr(t):
    return None if t is None else t.data_ptr()


def qmv_norm_rope_append(qkv: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, axis_of_pair,
                         slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         q_norm: torch.Tensor | None, k_norm: torch.Tensor | None, eps: float = 1e-6,
                         interleaved: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qmv_rope_append with an RMS norm of each q and k head before it is turned, weights
    q_norm and k_norm fp32 [D] (None: no norm)."""
    pages, page, Hkv, D = k_cache.shape
    M, dtype = qkv.shape[0], k_cache.dtype
    t = _type(k_cache, "k_cache", _16BIT)
    dev, Hq, axis_of_pair = _rope_args(qkv, positions, table, axis_of_pair, slots, k_cache, v_cache, q_norm, k_norm, dtype)
    if out is None:
        out = _empty((M, Hq, D), dtype, qkv.device, stream)
    else:
        _is(out, "out", dtype, (M, Hq, D), dev)
    status = _fn("qmv_norm_rope_append")(
        qkv.data_ptr(), positions.data_ptr(), table.data_ptr(), axis_of_pair, slots.data_ptr(), _ptr(q_norm), _ptr(k_norm),
        eps, out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), t, 1 if interleaved else 0, M, Hq, Hkv, D,
        2 * len(axis_of_pair), positions.shape[0], table.shape[0], pages * page, _on(stream, dev))
    if status != QMV_OK:
        _check("qmv_norm_rope_append", status)
    return out


def qmv_rope_append_e4m3(qkv: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, axis_of_pair,
                         slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None,
                         eps: float = 1e-6, interleaved: bool = False, dtype: torch.dtype = torch.float16,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The same into a cache of 8-bit codes: k_cache, v_cache float8_e4m3fn [pages, page, Hkv, D]
    with scales k_scale, v_scale fp32 [pages, page / 16, Hkv] of blocks of 16 slots, which
    grow with what is appended (rows of one block follow one another, in the slots' order).
    Returns q [M, Hq, D], fp16 or bf16 (dtype, or out's)."""
    pages, page, Hkv, D = k_cache.shape
    M = qkv.shape[0]
    dev, Hq, axis_of_pair = _rope_args(qkv, positions, table, axis_of_pair, slots, k_cache, v_cache, q_norm, k_norm, _E4M3)
    _is(k_scale, "k_scale", _F32, (pages, page // 16, Hkv), dev)
    _is(v_scale, "v_scale", _F32, (pages, page // 16, Hkv), dev)
    if page % 16 != 0:
        raise ValueError(f"k_cache: pages of {page} are not whole blocks of 16")
    if out is None:
        if dtype not in _16BIT:
            raise TypeError(f"dtype: expected {_F16} or {_BF16}, got {dtype}")
        out = _empty((M, Hq, D), dtype, qkv.device, stream)
    else:
        _type(out, "out", _16BIT)
        _is(out, "out", out.dtype, (M, Hq, D), dev)
    status = _fn("qmv_rope_append_e4m3")(
        qkv.data_ptr(), positions.data_ptr(), table.data_ptr(), axis_of_pair, slots.data_ptr(), _ptr(q_norm), _ptr(k_norm),
        eps, out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        _TYPE[out.dtype], 1 if interleaved else 0, M, Hq, Hkv, D, 2 * len(axis_of_pair), positions.shape[0],
        table.shape[0], pages * page, _on(stream, dev))
    if status != QMV_OK:
        _check("qmv_rope_append_e4m3", status)
    return out


def qmv_paged_attention_e4m3_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    """Bytes of workspace of qmv_paged_attention_e4m3 at these sizes."""
    return _bytes("qmv_paged_attention_e4m3_workspace",
                  _fn("qmv_paged_attention_e4m3_workspace")(B, T, Hq, Hkv, D, max_len))


def qmv_paged_attention_e4m3(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                             v_scale: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, scale: float | None = None,
                             max_len: int | None = None, out: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of q [B, T, Hq, D], the last T of each request's lens[b] tokens (int32 [B]),
    over the pages table[b] (int32 [B, n]) of a cache of codes as qmv_rope_append_e4m3 fills
    it. scale: 1 / sqrt(D) unless given. max_len: a bound of lens that the caller knows (the
    table's width unless given; the work is split by it)."""
    B, T, Hq, D = q.shape
    pages, page, Hkv, _ = k_cache.shape
    width = table.shape[1]
    dtype = q.dtype
    t = _type(q, "q", _16BIT)
    dev = _first(q, "q", dtype)
    _is(k_cache, "k_cache", _E4M3, (pages, page, Hkv, D), dev)
    _is(v_cache, "v_cache", _E4M3, k_cache.shape, dev)
    _is(k_scale, "k_scale", _F32, (pages, page // 16, Hkv), dev)
    _is(v_scale, "v_scale", _F32, k_scale.shape, dev)
    _is(table, "table", _I32, (B, width), dev)
    _is(lens, "lens", _I32, (B,), dev)
    if max_len is None:
        max_len = width * page
    if out is None:
        out = _empty((B, T, Hq, D), dtype, q.device, stream)
    else:
        _is(out, "out", dtype, q.shape, dev)
    need = lambda: qmv_paged_attention_e4m3_workspace(B, T, Hq, Hkv, D, max_len)  # noqa: E731
    ws = _workspace(workspace, need, dev, stream)
    status = _fn("qmv_paged_attention_e4m3")(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), t, pages, page,
        table.data_ptr(), width, lens.data_ptr(), max_len, 1.0 / math.sqrt(D) if scale is None else scale, out.data_ptr(),
        ws.data_ptr(), ws.numel(), B, T, Hq, Hkv, D, _on(stream, dev))
    if status != QMV_OK:
        _check_with("qmv_paged_attention_e4m3", status, ws, need)
    return out


def qmv_prefix_attention_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, prefix_len: int, max_own: int) -> int:
    """Bytes of workspace of qmv_prefix_attention at these sizes."""
    return _bytes("qmv_prefix_attention_workspace",
                  _fn("qmv_prefix_attention_workspace")(B, T, Hq, Hkv, D, prefix_len, max_own))


def qmv_prefix_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, prefix_table: torch.Tensor,
                         prefix_len: int, own_table: torch.Tensor, own_len: torch.Tensor, scale: float | None = None,
                         max_own: int | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of q [B, T, Hq, D] over a prefix that all requests share (prefix_len keys
    in the pages prefix_table int32 [n]) and each request's own_len[b] own keys (int32 [B],
    in the pages own_table[b] int32 [B, own_pages]), its T tokens being the last of them;
    k_cache, v_cache [pages, page, Hkv, D]. scale: 1 / sqrt(D) unless given. max_own: a
    bound of own_len that the caller knows (the table's width unless given; the work is
    split by it)."""
    B, T, Hq, D = q.shape
    pages, page, Hkv, _ = k_cache.shape
    own_pages = own_table.shape[1]
    dtype = q.dtype
    t = _type(q, "q", _16BIT)
    dev = _first(q, "q", dtype)
    _is(k_cache, "k_cache", dtype, (pages, page, Hkv, D), dev)
    _is(v_cache, "v_cache", dtype, k_cache.shape, dev)
    _held(prefix_table, "prefix_table", _I32, dev)
    _is(own_table, "own_table", _I32, (B, own_pages), dev)
    _is(own_len, "own_len", _I32, (B,), dev)
    if prefix_table.numel() * page < prefix_len:
        raise ValueError(f"prefix_table: {prefix_table.numel()} pages of {page} hold no {prefix_len} keys")
    if max_own is None:
        max_own = own_pages * page
    if out is None:
        out = _empty((B, T, Hq, D), dtype, q.device, stream)
    else:
        _is(out, "out", dtype, q.shape, dev)
    need = lambda: qmv_prefix_attention_workspace(B, T, Hq, Hkv, D, prefix_len, max_own)  # noqa: E731
    ws = _workspace(workspace, need, dev, stream)
    status = _fn("qmv_prefix_attention")(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), t, pages, page, prefix_table.data_ptr(), prefix_len,
        own_table.data_ptr(), own_pages, own_len.data_ptr(), max_own, 1.0 / math.sqrt(D) if scale is None else scale,
        out.data_ptr(), ws.data_ptr(), ws.numel(), B, T, Hq, Hkv, D, _on(stream, dev))
    if status != QMV_OK:
        _check_with("qmv_prefix_attention", status, ws, need)
    return out


def qmv_penalize_logits(logits: torch.Tensor, tokens: torch.Tensor, prompt_len: torch.Tensor, total_len: torch.Tensor,
                        repetition: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                        frequency: torch.Tensor | None = None, bias_tokens: torch.Tensor | None = None,
                        bias_values: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                        mask_row: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Penalties for the tokens of each row's history, biases and masks on logits fp32
    [M, V]: tokens int32 [M, H], of which the first total_len[m] count (the first
    prompt_len[m] are the prompt's); repetition, presence, frequency fp32 [M] or None;
    bias_tokens int32 and bias_values fp32 [M, n]; mask int32 [n_masks, ceil(V/32)], bit
    set = allowed, with mask_row int32 [M] (negative: none). out may be logits."""
    M, V = logits.shape
    H = tokens.shape[1]
    dev = _first(logits, "logits", _F32)
    _is(tokens, "tokens", _I32, (M, H), dev)
    _is(prompt_len, "prompt_len", _I32, (M,), dev)
    _is(total_len, "total_len", _I32, (M,), dev)
    rows = []
    for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
        if t is not None:
            _is(t, name, _F32, (M,), dev)
        rows.append(None if t is None else t.data_ptr())
    n_bias = n_masks = 0
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values come together")
    if bias_tokens is not None:
        n_bias = bias_tokens.shape[1]
        _is(bias_tokens, "bias_tokens", _I32, (M, n_bias), dev)
        _is(bias_values, "bias_values", _F32, (M, n_bias), dev)
    if mask is not None:
        n_masks = mask.shape[0]
        _is(mask, "mask", _I32, (n_masks, (V + 31) // 32), dev)
    if mask_row is not None:
        _is(mask_row, "mask_row", _I32, (M,), dev)
    if out is None:
        out = _empty((M, V), _F32, logits.device, stream)
    else:
        _is(out, "out", _F32, (M, V), dev)
    status = _fn("qmv_penalize_logits")(
        logits.data_ptr(), tokens.data_ptr(), H, prompt_len.data_ptr(), total_len.data_ptr(), *rows,
        None if bias_tokens is None else bias_tokens.data_ptr(), None if bias_values is None else bias_values.data_ptr(),
        n_bias, None if mask is None else mask.data_ptr(), None if mask_row is None else mask_row.data_ptr(), n_masks,
        out.data_ptr(), M, V, _on(stream, dev))
    if status != QMV_OK:
        _check("qmv_penalize_logits", status)
    return out


def qmv_sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
               top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None,
               out: torch.Tensor | None = None, prob: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """A token int32 for each row of logits fp32 [M, V], drawn by the random numbers u fp32 [M],
    0 <= u < 1, among those that top_k int32, top_p and min_p fp32 [M] keep (None: all), at
    temperature fp32 [M] (None: 1; 0: the largest logit). prob fp32 [M], where given, gets the
    token's probability among those kept. A row without a logit above -inf gives -1."""
    M, V = logits.shape
    dev = _first(logits, "logits", _F32)
    _is(u, "u", _F32, (M,), dev)
    for name, t, dtype in (("temperature", temperature, _F32), ("top_k", top_k, _I32), ("top_p", top_p, _F32),
                           ("min_p", min_p, _F32), ("prob", prob, _F32)):
        if t is not None:
            _is(t, name, dtype, (M,), dev)
    if out is None:
        out = _empty((M,), _I32, logits.device, stream)
    else:
        _is(out, "out", _I32, (M,), dev)
    status = _fn("qmv_sample")(logits.data_ptr(), u.data_ptr(), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
                               out.data_ptr(), _ptr(prob), M, V, _on(stream, dev))
    if status != QMV_OK:
        _check("qmv_sample", status)
    return out
