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

Weights and prompts are synthetic. ``python -m gemm_qmv_quantize_gb300.decode_step`` times
each call on the 27B-class shapes (hidden 5120, 40 query heads over 8 key heads of 128,
vocabulary 151936), with 32 requests behind a prompt of 8192 tokens.
"""
from __future__ import annotations

import argparse
import math

import torch

from . import (qgemm_nvfp4_w4a16, qmv_lora_add, qmv_lora_add_workspace, qmv_penalize_logits, qmv_prefix_attention,
               qmv_prefix_attention_workspace, qmv_rope_append, qmv_rope_table, synth)


class DecodeStep:
    """Weights, cache and workspaces of the step. The cache's first pages hold the prompt
    (written by one qmv_rope_append over its tokens), then each request has pages of its own,
    for max_own tokens: as many steps can be taken. (A step replayed from a CUDA graph is not
    counted here; one too many takes the last token's place and sets bit 2 of error_flags.)"""

    def __init__(self, batch: int, prefix_len: int, max_own: int, hidden: int = 5120, Hq: int = 40, Hkv: int = 8,
                 D: int = 128, vocab: int = 151936, adapters: int = 8, rank: int = 16, page: int = 64, seed: int = 0,
                 device="cuda"):
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
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=torch.float16, device=device) for _ in range(2))
        pages = torch.arange(shape[0], dtype=torch.int32, device=device)
        self.prefix_table = pages[:n_prefix].contiguous()
        self.own_table = pages[n_prefix:].reshape(batch, n_own).contiguous()
        self.own_len = torch.zeros((batch,), dtype=torch.int32, device=device)
        self.table = qmv_rope_table(prefix_len + max_own, D, 1e6, device)
        self.axes = bytes(D // 2)   # text: one axis
        prompt = normal(prefix_len, qkv)
        at = torch.arange(prefix_len, device=device)
        qmv_rope_append(prompt, at.to(torch.int32)[None].contiguous(), self.table, self.axes, at, self.k_cache, self.v_cache)
        # what is known of the answers so far
        self.tokens = torch.full((batch, max_own), -1, dtype=torch.int32, device=device)
        self.prompt_len = torch.zeros((batch,), dtype=torch.int32, device=device)
        self.repetition = torch.full((batch,), 1.1, device=device)
        self.presence = torch.full((batch,), 0.2, device=device)
        self.frequency = torch.full((batch,), 0.1, device=device)
        self.mask = torch.randint(-2 ** 31, 2 ** 31, (1, (vocab + 31) // 32), generator=g, device=device).to(torch.int32)
        self.mask_row = torch.where(torch.arange(batch, device=device) % 2 == 0, 0, -1).to(torch.int32)
        bytes_ = max(qmv_lora_add_workspace(batch, rank, max(hidden, Hq * D)),
                     qmv_prefix_attention_workspace(batch, 1, Hq, Hkv, D, prefix_len, max_own))
        self.workspace = torch.empty((bytes_,), dtype=torch.uint8, device=device)   # of one call at a time

    def project(self, name: str, x: torch.Tensor) -> torch.Tensor:
        y = qgemm_nvfp4_w4a16(*self.w[name], x)
        return qmv_lora_add(x, self.a[name], self.b[name], self.adapter, self.scale, y, out=y, workspace=self.workspace)

    def step(self, x: torch.Tensor, timed=lambda name, f: f()) -> dict:
        """x fp16 [batch, hidden]: the state of each request's newest token. Returns what
        each call made; the logits under "logits". timed(name, call) runs each call."""
        if self.taken >= self.max_own:
            raise ValueError(f"{self.taken} steps taken: the requests have room for {self.max_own} tokens of their own")
        self.taken += 1
        at = self.own_len.clamp(max=self.max_own - 1).long()
        own_slot = self.own_table.gather(1, (at // self.page)[:, None])[:, 0].long() * self.page + at % self.page
        position = (self.own_len + self.prefix_len)[None].contiguous()
        qkv = timed("qkv projection + adapters", lambda: self.project("qkv", x))
        q = timed("rotary + append", lambda: qmv_rope_append(qkv, position, self.table, self.axes, own_slot, self.k_cache,
                                                             self.v_cache))
        self.own_len += 1
        o = timed("attention", lambda: qmv_prefix_attention(
            q.view(self.B, 1, self.Hq, self.D), self.k_cache, self.v_cache, self.prefix_table, self.prefix_len,
            self.own_table, self.own_len, max_own=self.max_own, workspace=self.workspace)).view(self.B, -1)
        hidden = timed("o projection + adapters", lambda: self.project("o", o))
        raw = timed("output head", lambda: qgemm_nvfp4_w4a16(*self.w["head"], hidden.half()))
        logits = timed("penalties and masks", lambda: qmv_penalize_logits(
            raw, self.tokens, self.prompt_len, at.to(torch.int32), self.repetition, self.presence, self.frequency,
            mask=self.mask, mask_row=self.mask_row))
        self.tokens.scatter_(1, at[:, None], logits.argmax(1, keepdim=True).to(torch.int32))
        return {"qkv": qkv, "q": q, "o": o, "hidden": hidden, "raw": raw, "logits": logits}


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--batch", type=int, default=32)
    p.add_argument("--prefix", type=int, default=8192)
    p.add_argument("--max-own", type=int, default=512)
    p.add_argument("--steps", type=int, default=20)
    args = p.parse_args()
    if not 3 < args.steps <= args.max_own:
        p.error(f"--steps: more than the 3 of the warm-up and at most --max-own ({args.max_own})")
    net = DecodeStep(args.batch, args.prefix, args.max_own)
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
        net.step(x, timed)
    torch.cuda.synchronize()
    for name, pairs in times.items():
        us = sorted(a.elapsed_time(b) * 1e3 for a, b in pairs[3:])
        print(f"{name:28s} {us[len(us) // 2]:8.1f} us (median of {len(us)})")


if __name__ == "__main__":
    main()
