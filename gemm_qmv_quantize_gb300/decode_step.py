"""A batched decode step that runs the operators beside the quantized matmuls together.

Requests share a long prompt and go on with tokens of their own, each with its adapter. A
step takes one hidden state a request through an attention block and the output head:

    q|k|v  = NVFP4 projection              qgemm_nvfp4_w4a16
           + the requests' adapters        qmv_lora_add (in place)
    q, cache = rotary positions, append    qmv_rope_append
    o      = prefix and own tokens         qmv_prefix_attention
    hidden = NVFP4 projection + adapters   qgemm_nvfp4_w4a16, qmv_lora_add
    logits = NVFP4 output head             qgemm_nvfp4_w4a16
             penalties, grammar masks      qmv_penalize_logits
    token  = the largest logit, or a draw  qmv_sample

With norms, each q and k head has an RMS norm before its position (qmv_norm_rope_append); with
a cache of 8 bits, the append writes E4M3 codes and their scales (qmv_rope_append_e4m3) and
qmv_paged_attention_e4m3 reads them, the prompt's pages standing in every request's page table.

Weights and prompts are synthetic. ``python -m gemm_qmv_quantize_gb300.decode_step`` times
each call on the 27B-class shapes (hidden 5120, 40 query heads over 8 key heads of 128,
vocabulary 151936), with 32 requests behind a prompt of 8192 tokens.
"""
from __future__ import annotations

import argparse
import math

import torch

from . import (qgemm_nvfp4_w4a16, qmv_lora_add, qmv_lora_add_workspace, qmv_norm_rope_append, qmv_paged_attention_e4m3,
               qmv_paged_attention_e4m3_workspace, qmv_penalize_logits, qmv_prefix_attention,
               qmv_prefix_attention_workspace, qmv_rope_append, qmv_rope_append_e4m3, qmv_rope_table, qmv_sample, synth)


class DecodeStep:
    """Weights, cache and workspaces of the step. The cache's first pages hold the prompt
    (written by one qmv_rope_append over its tokens), then each request has pages of its own,
    for max_own tokens: as many steps can be taken. (A step replayed from a CUDA graph is not
    counted here; one too many takes the last token's place and sets bit 2 of error_flags.)"""

    def __init__(self, batch: int, prefix_len: int, max_own: int, hidden: int = 5120, Hq: int = 40, Hkv: int = 8,
                 D: int = 128, vocab: int = 151936, adapters: int = 8, rank: int = 16, page: int = 64, seed: int = 0,
                 device="cuda", norms: bool = False, cache: str = "f16"):
        if cache not in ("f16", "e4m3"):
            raise ValueError(f"cache: f16 or e4m3, not {cache}")
        if cache == "e4m3" and prefix_len % page:
            raise ValueError(f"prefix_len: {prefix_len} tokens do not end with a page of {page}, as a page table with the prompt's pages wants")
        self.taken = 0   # steps
        self.B, self.prefix_len, self.max_own, self.Hq, self.Hkv, self.D, self.page = batch, prefix_len, max_own, Hq, Hkv, D, page
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        qkv = (Hq + 2 * Hkv) * D
        # codes, group scales and the tensor scale of each projection
        self.w = {name: synth.nvfp4_weights(n, k, seed=seed + i + 1, device=device)
                  for i, (name, n, k) in enumerate((("qkv", qkv, hidden), ("o", hidden, Hq * D), ("head", vocab, hidden)))}
        self.a = {n: (normal(adapters, rank, k) / math.sqrt(k)).half() for n, k in (("qkv", hidden), ("o", Hq * D))}
        self.b = {n: (normal(adapters, m, rank) / math.sqrt(rank)).half() for n, m in (("qkv", qkv), ("o", hidden))}
        self.scale = torch.full((adapters,), 0.5, device=device)
        self.adapter = torch.randint(-1, adapters, (batch,), generator=g, device=device, dtype=torch.int32)
        # caches and page tables
        n_prefix, n_own = -(-prefix_len // page), -(-max_own // page)
        shape = (n_prefix + batch * n_own, page, Hkv, D)
        self.cache8 = cache == "e4m3"
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=torch.float8_e4m3fn if self.cache8 else torch.float16, device=device)
                                      for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones((shape[0], page // 16, Hkv), device=device) for _ in range(2)) if self.cache8 else (None, None)
        pages = torch.arange(shape[0], dtype=torch.int32, device=device)
        self.prefix_table = pages[:n_prefix].contiguous()
        self.own_table = pages[n_prefix:].reshape(batch, n_own).contiguous()
        self.own_len = torch.zeros((batch,), dtype=torch.int32, device=device)
        self.table = qmv_rope_table(prefix_len + max_own, D, 1e6, device)
        self.axes = bytes(D // 2)   # text: one axis
        prompt = normal(prefix_len, qkv)
        at = torch.arange(prefix_len, device=device)
        weights = torch.Generator(device=device).manual_seed(seed + 1000)
        self.q_norm, self.k_norm = (torch.rand((D,), generator=weights, device=device) + 0.5 for _ in range(2)) if norms else (None, None)
        self.append(prompt, at.to(torch.int32)[None].contiguous(), at)
        self.page_table = torch.cat([self.prefix_table.expand(batch, -1), self.own_table], 1).contiguous()   # of all tokens
        # what is known of the answers so far
        self.tokens = torch.full((batch, max_own), -1, dtype=torch.int32, device=device)
        self.prompt_len = torch.zeros((batch,), dtype=torch.int32, device=device)
        self.repetition = torch.full((batch,), 1.1, device=device)
        self.presence = torch.full((batch,), 0.2, device=device)
        self.frequency = torch.full((batch,), 0.1, device=device)
        self.mask = torch.randint(-2 ** 31, 2 ** 31, (1, (vocab + 31) // 32), generator=g, device=device).to(torch.int32)
        self.mask_row = torch.where(torch.arange(batch, device=device) % 2 == 0, 0, -1).to(torch.int32)
        self.temperature = torch.full((batch,), 0.8, device=device)
        self.top_k = torch.full((batch,), 50, dtype=torch.int32, device=device)
        self.top_p = torch.full((batch,), 0.95, device=device)
        self.min_p = torch.full((batch,), 0.02, device=device)
        bytes_ = max(qmv_lora_add_workspace(batch, rank, max(hidden, Hq * D)),
                     qmv_paged_attention_e4m3_workspace(batch, 1, Hq, Hkv, D, prefix_len + max_own) if self.cache8 else
                     qmv_prefix_attention_workspace(batch, 1, Hq, Hkv, D, prefix_len, max_own))
        self.workspace = torch.empty((bytes_,), dtype=torch.uint8, device=device)   # of one call at a time

    def project(self, name: str, x: torch.Tensor) -> torch.Tensor:
        y = qgemm_nvfp4_w4a16(*self.w[name], x)
        return qmv_lora_add(x, self.a[name], self.b[name], self.adapter, self.scale, y, out=y, workspace=self.workspace)

    def append(self, qkv: torch.Tensor, position: torch.Tensor, slots: torch.Tensor) -> torch.Tensor:
        if self.cache8:
            return qmv_rope_append_e4m3(qkv, position, self.table, self.axes, slots, self.k_cache, self.v_cache, self.k_scale,
                                        self.v_scale, self.q_norm, self.k_norm)
        if self.q_norm is not None:
            return qmv_norm_rope_append(qkv, position, self.table, self.axes, slots, self.k_cache, self.v_cache, self.q_norm,
                                        self.k_norm)
        return qmv_rope_append(qkv, position, self.table, self.axes, slots, self.k_cache, self.v_cache)

    def attend(self, q: torch.Tensor) -> torch.Tensor:
        q = q.view(self.B, 1, self.Hq, self.D)
        if self.cache8:
            return qmv_paged_attention_e4m3(q, self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.page_table,
                                            self.own_len + self.prefix_len, max_len=self.prefix_len + self.max_own,
                                            workspace=self.workspace)
        return qmv_prefix_attention(q, self.k_cache, self.v_cache, self.prefix_table, self.prefix_len, self.own_table,
                                    self.own_len, max_own=self.max_own, workspace=self.workspace)

    def step(self, x: torch.Tensor, timed=lambda name, f: f(), u: torch.Tensor | None = None) -> dict:
        """x fp16 [batch, hidden]: the state of each request's newest token. Returns what
        each call made; the logits under "logits", the tokens under "token". timed(name, call) runs
        each call. u fp32 [batch], random numbers of 0 <= u < 1: tokens are drawn, else those of the
        largest logits."""
        if self.taken >= self.max_own:
            raise ValueError(f"{self.taken} steps taken: the requests have room for {self.max_own} tokens of their own")
        self.taken += 1
        at = self.own_len.clamp(max=self.max_own - 1).long()
        own_slot = self.own_table.gather(1, (at // self.page)[:, None])[:, 0].long() * self.page + at % self.page
        position = (self.own_len + self.prefix_len)[None].contiguous()
        qkv = timed("qkv projection + adapters", lambda: self.project("qkv", x))
        q = timed("rotary + append", lambda: self.append(qkv, position, own_slot))
        self.own_len += 1
        o = timed("attention", lambda: self.attend(q)).view(self.B, -1)
        hidden = timed("o projection + adapters", lambda: self.project("o", o))
        raw = timed("output head", lambda: qgemm_nvfp4_w4a16(*self.w["head"], hidden.half()))
        logits = timed("penalties and masks", lambda: qmv_penalize_logits(
            raw, self.tokens, self.prompt_len, at.to(torch.int32), self.repetition, self.presence, self.frequency,
            mask=self.mask, mask_row=self.mask_row))
        if u is None:
            token = logits.argmax(1).to(torch.int32)
        else:
            token = timed("sampling", lambda: qmv_sample(logits, u, self.temperature, self.top_k, self.top_p, self.min_p))
        self.tokens.scatter_(1, at[:, None], token[:, None])
        return {"qkv": qkv, "q": q, "o": o, "hidden": hidden, "raw": raw, "logits": logits, "token": token}


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--batch", type=int, default=32)
    p.add_argument("--prefix", type=int, default=8192)
    p.add_argument("--max-own", type=int, default=512)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--cache", choices=("f16", "e4m3"), default="f16")
    p.add_argument("--norms", action="store_true", help="norms of q and k heads")
    p.add_argument("--sample", action="store_true", help="draw tokens instead of the largest logits")
    args = p.parse_args()
    if not 3 < args.steps <= args.max_own:
        p.error(f"--steps: more than the 3 of the warm-up and at most --max-own ({args.max_own})")
    if args.cache == "e4m3" and args.prefix % 64:
        p.error(f"--prefix: a multiple of the pages' 64 tokens with --cache e4m3, not {args.prefix}")
    net = DecodeStep(args.batch, args.prefix, args.max_own, **({"norms": True} if args.norms else {}),
                     **({"cache": args.cache} if args.cache != "f16" else {}))
    u = torch.rand((args.batch,), device="cuda") if args.sample else None
    x = torch.randn((args.batch, 5120), device="cuda").half()
    times = {}

    def timed(name, call):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        r = call()
        end.record()
        times.setdefault(name, []).append((start, end))
        return r

    for _ in range(args.steps):
        net.step(x, timed, **({} if u is None else {"u": u}))
    torch.cuda.synchronize()
    for name, pairs in times.items():
        us = sorted(a.elapsed_time(b) * 1e3 for a, b in pairs[3:])
        print(f"{name:28s} {us[len(us) // 2]:8.1f} us (median of {len(us)})")


if __name__ == "__main__":
    main()
