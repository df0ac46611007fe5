"""The operators of a batched decode step that stand beside the quantized matmuls.

- ``lora``: low-rank adapters of many requests, added to a shared projection's output.
- ``rope``: rotary positions with one to three axes on the projection's q and k, and the
  append of k and v to a paged cache.
- ``attention``: attention of a batch whose requests share a long prefix and go on with
  tokens of their own, both in the paged cache.
- ``logits``: penalties for repeated tokens, biases and grammar masks on the logits.

``listed`` names fixed cases, ``draw`` makes one of the same ranges, ``prepare`` makes a
case's inputs, ``run`` computes one pass (the plain form in 32 bits, or the library's calls
where ``own`` is true), ``exact`` the same in 64 bits and ``work`` counts the bytes and
operations that a pass cannot do without.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def lora(name, M, N, K, R, adapters, x, w, spread):
    """spread: "each" (every row another adapter), "shared" (all rows one), "mixed"
    (drawn, with some rows that have none)."""
    return {"name": name, "op": "lora", "M": M, "N": N, "K": K, "R": R, "adapters": adapters, "x": x, "w": w,
            "spread": spread}


def rope(name, M, Hq, Hkv, D, rot, axes, interleaved, type_, positions):
    return {"name": name, "op": "rope", "M": M, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "axes": axes,
            "interleaved": interleaved, "type": type_, "positions": positions}


def attention(name, B, T, Hq, Hkv, D, prefix, own_max, page, type_):
    return {"name": name, "op": "attention", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "prefix": prefix,
            "own_max": own_max, "page": page, "type": type_}


def logits(name, M, V, history, biases, masks):
    return {"name": name, "op": "logits", "M": M, "V": V, "history": history, "biases": biases, "masks": masks}


def listed():
    return [
        # one request's adapter beside a 4096 x 4096 projection: latency counts
        lora("lora_one_token", 1, 4096, 4096, 16, 4, "f16", "f16", "each"),
        # eight rows of fp32 activations (the Q4_0 path) beside a 14336 x 4096 projection, few adapters
        lora("lora_eight_rows", 8, 14336, 4096, 32, 6, "f32", "bf16", "mixed"),
        # a full batch of 96 rows, an adapter each, beside a 17408 x 5120 projection
        lora("lora_full_batch", 96, 17408, 5120, 64, 96, "f16", "bf16", "each"),
        # one token of a decode step, one position axis, as many key heads as query heads
        rope("rope_one_token", 1, 32, 32, 128, 128, 1, False, "f16", 4096),
        # the tokens of an image in a prompt: three axes, 40 query heads over 8 key heads
        rope("rope_image_prompt", 4001, 40, 8, 128, 128, 3, False, "bf16", 32768),
        # one request alone with a short prefix: latency counts
        attention("attention_one_request", 1, 1, 32, 8, 128, 500, 60, 16, "f16"),
        # an ordinary batch behind a system prompt
        attention("attention_batch", 24, 1, 40, 8, 128, 8191, 700, 64, "bf16"),
        # speculative verification: 5 tokens of each request, 64-wide heads
        attention("attention_verify", 16, 5, 32, 4, 64, 4099, 333, 32, "f16"),
        # a full batch behind a long shared document
        attention("attention_long_prefix", 64, 1, 40, 8, 128, 65536, 1024, 64, "bf16"),
        # one row of a small vocabulary: latency counts
        logits("logits_one_row", 1, 32000, 200, 0, 0),
        # eight long conversations over a large vocabulary
        logits("logits_long_history", 8, 151936, 16000, 100, 0),
        # a full batch, most of it under a grammar
        logits("logits_full_batch", 96, 151936, 3000, 60, 80),
    ]


def spread_over(rng, low, high):
    """A whole number of low..high, even over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["lora", "rope", "attention", "logits"])
    if op == "lora":
        # everything up to the largest listed case, which reads the weights of 96 adapters
        M, R = spread_over(rng, 1, 96), 8 * spread_over(rng, 1, 16)
        N, K = spread_over(rng, 64, 17408), 8 * spread_over(rng, 8, 2176)
        while M * R * (N + K) > 96 * 64 * (17408 + 5120):
            N, K = max(1, N // 2), max(8, K // 16 * 8)
        c = lora("", M, N, K, R, spread_over(rng, 1, 96), rng.choice(["f16", "f32"]), rng.choice(["f16", "bf16"]),
                 rng.choice(["each", "shared", "mixed"]))
    elif op == "rope":
        D, Hkv = rng.choice([64, 80, 128, 256]), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.randint(1, 8)
        M = spread_over(rng, 1, 4001)
        while M * (Hq + 2 * Hkv) * D > 4001 * 56 * 128:
            M //= 2
        c = rope("", M, Hq, Hkv, D, rng.choice([D, D, D // 2]), rng.choice([1, 3]), rng.random() < 0.4,
                 rng.choice(["f16", "bf16"]), spread_over(rng, 4096, 65536))
    elif op == "attention":
        B, T, D = spread_over(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8]), rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.randint(1, 8)
        prefix, own_max = spread_over(rng, 1, 65536), max(T, spread_over(rng, 1, 2048))
        while B * T * Hq * prefix * D > 64 * 40 * 65536 * 128:
            prefix //= 2
        while B * own_max * Hkv * D > 64 * 1024 * 8 * 128:
            own_max = max(T, own_max // 2)
        c = attention("", B, T, Hq, Hkv, D, prefix, own_max, rng.choice([16, 32, 64, 128]), rng.choice(["f16", "bf16"]))
    else:
        M, V = spread_over(rng, 1, 96), spread_over(rng, 1000, 151936)
        history = spread_over(rng, 1, 16000)
        while M * history > 96 * 3000:
            history //= 2
        c = logits("", M, V, history, rng.choice([0, 0, 1, 40, 300]), rng.choice([0, M, (M + 1) // 2]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 7919 + 17)
    return {"lora": prepare_lora, "rope": prepare_rope, "attention": prepare_attention,
            "logits": prepare_logits}[case["op"]](case, g)


def normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * scale).to(dtype)


def whole(g, low, high, shape, dtype=torch.int32):
    return torch.randint(low, high, shape, generator=g, device=DEVICE, dtype=dtype)


def prepare_lora(c, g):
    M, N, K, R, L = (c[k] for k in ("M", "N", "K", "R", "adapters"))
    if c["spread"] == "each":
        adapter = (torch.randperm(max(M, L), generator=g, device=DEVICE)[:M] % L).to(torch.int32)
    elif c["spread"] == "shared":
        adapter = torch.full((M,), L - 1, dtype=torch.int32, device=DEVICE)
    else:
        adapter = whole(g, -1, L, (M,))
    w = TYPES[c["w"]]
    return {"op": "lora", "adapter": adapter,
            "x": normal(g, (M, K), TYPES[c["x"]]),
            "base": normal(g, (M, N)),                       # the shared projection's output
            "a": normal(g, (L, R, K), w, 1 / math.sqrt(K)),
            "b": normal(g, (L, N, R), w, 0.5 / math.sqrt(R)),
            "scale": torch.rand((L,), generator=g, device=DEVICE) + 0.5,
            "out": torch.empty((M, N), device=DEVICE),
            "workspace": {}}


def rope_sections(pairs, axes):
    """The axis of each pair, by the common rule: time the first quarter, then height and
    width three eighths each."""
    if axes == 1:
        return [0] * pairs
    t, h = pairs // 4, (pairs * 3) // 8
    return [0 if i < t else 1 if i < t + h else 2 for i in range(pairs)]


def prepare_rope(c, g):
    M, Hq, Hkv, D, rot, A = (c[k] for k in ("M", "Hq", "Hkv", "D", "rot", "axes"))
    pairs, dtype = rot // 2, TYPES[c["type"]]
    inv = 1e6 ** -(torch.arange(pairs, dtype=torch.float64, device=DEVICE) / pairs)
    angle = torch.arange(c["positions"], dtype=torch.float64, device=DEVICE)[:, None] * inv
    page = 16
    pages = (2 * M + 64 + page - 1) // page
    # a cache of twice the tokens, whose free slots the tokens take in no order; one in 16 is padding
    slots = torch.randperm(pages * page, generator=g, device=DEVICE)[:M].to(torch.int64)
    if M > 1:
        slots = torch.where(torch.rand((M,), generator=g, device=DEVICE) < 1 / 16, torch.full_like(slots, -1), slots)
    return {"op": "rope", "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "interleaved": c["interleaved"],
            "axis_of_pair": bytes(rope_sections(pairs, A)),
            "axis": torch.tensor(rope_sections(pairs, A), device=DEVICE),
            "qkv": normal(g, (M, (Hq + 2 * Hkv) * D)),       # the shared projection's output
            "positions": whole(g, 0, c["positions"], (A, M)),
            "table": torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32).contiguous(),
            "slots": slots,
            "k_cache": normal(g, (pages, page, Hkv, D), dtype), "v_cache": normal(g, (pages, page, Hkv, D), dtype),
            "q": torch.empty((M, Hq, D), dtype=dtype, device=DEVICE)}


def prepare_attention(c, g):
    B, T, Hq, Hkv, D, prefix, own_max, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "prefix", "own_max", "page"))
    dtype = TYPES[c["type"]]
    n_prefix, n_own = (prefix + page - 1) // page, (own_max + page - 1) // page
    pages = n_prefix + B * n_own + 3
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)   # pages lie in no order
    own_len = whole(g, T, own_max + 1, (B,))
    own_len[0] = own_max
    return {"op": "attention", "prefix_len": prefix, "max_own": own_max, "scale": 1 / math.sqrt(D),
            "q": normal(g, (B, T, Hq, D), dtype, 1.5),
            "k_cache": normal(g, (pages, page, Hkv, D), dtype), "v_cache": normal(g, (pages, page, Hkv, D), dtype),
            "prefix_table": order[:n_prefix].contiguous(),
            "own_table": order[n_prefix:n_prefix + B * n_own].reshape(B, n_own).contiguous(),
            "own_len": own_len,
            "out": torch.empty((B, T, Hq, D), dtype=dtype, device=DEVICE),
            "workspace": {}}


def prepare_logits(c, g):
    M, V, H, nb, nm = (c[k] for k in ("M", "V", "history", "biases", "masks"))
    total = whole(g, (H + 1) // 2, H + 1, (M,))
    total[0] = H
    # tokens of a text: few of them often, many rarely
    tokens = (V * torch.rand((M, H), generator=g, device=DEVICE) ** 3).to(torch.int32).clamp_(0, V - 1)
    state = {"op": "logits", "logits": normal(g, (M, V), scale=4.0), "tokens": tokens,
             "prompt_len": (total * torch.rand((M,), generator=g, device=DEVICE)).to(torch.int32), "total_len": total,
             "repetition": torch.rand((M,), generator=g, device=DEVICE) * 0.4 + 1.0,
             "presence": torch.rand((M,), generator=g, device=DEVICE),
             "frequency": torch.rand((M,), generator=g, device=DEVICE) * 0.5,
             "bias_tokens": None, "bias_values": None, "mask": None, "mask_row": None,
             "out": torch.empty((M, V), device=DEVICE)}
    if nb:
        n = min(nb, V)
        state["bias_tokens"] = torch.rand((M, V), generator=g, device=DEVICE).topk(n, dim=1).indices.to(torch.int32)
        state["bias_tokens"][torch.rand((M, n), generator=g, device=DEVICE) < 0.2] = -1   # rows have fewer than n
        state["bias_values"] = normal(g, (M, n), scale=3.0)
    if nm:
        state["mask"] = whole(g, -2**31, 2**31, (nm, (V + 31) // 32), torch.int64).to(torch.int32)
        row = torch.arange(M, device=DEVICE, dtype=torch.int32)
        state["mask_row"] = torch.where(row < nm, row, torch.full_like(row, -1))
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return OWN[state["op"]](state)
    return PLAIN[state["op"]](state)


def own_lora(s):
    import gemm_qmv_quantize_gb300 as q
    ws = kept(s, q.qmv_lora_add_workspace, s["x"].shape[0], s["a"].shape[1], s["x"].shape[1])
    return q.qmv_lora_add(s["x"], s["a"], s["b"], s["adapter"], s["scale"], s["base"], out=s["out"], workspace=ws)


def own_rope(s):
    import gemm_qmv_quantize_gb300 as q
    q.qmv_rope_append(s["qkv"], s["positions"], s["table"], s["axis_of_pair"], s["slots"], s["k_cache"], s["v_cache"],
                      interleaved=s["interleaved"], out=s["q"])
    return s["q"], s["k_cache"], s["v_cache"]


def own_attention(s):
    import gemm_qmv_quantize_gb300 as q
    ws = kept(s, q.qmv_prefix_attention_workspace, *s["q"].shape[:3], s["k_cache"].shape[2], s["q"].shape[3],
              s["prefix_len"], s["max_own"])
    return q.qmv_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_len"],
                                  s["own_table"], s["own_len"], scale=s["scale"], max_own=s["max_own"], out=s["out"],
                                  workspace=ws)


def own_logits(s):
    import gemm_qmv_quantize_gb300 as q
    return q.qmv_penalize_logits(s["logits"], s["tokens"], s["prompt_len"], s["total_len"], s["repetition"],
                                 s["presence"], s["frequency"], bias_tokens=s["bias_tokens"],
                                 bias_values=s["bias_values"], mask=s["mask"], mask_row=s["mask_row"], out=s["out"])


def kept(s, size, *sizes):
    """The workspace that a user's program keeps for calls of these sizes."""
    if "buffer" not in s["workspace"]:
        s["workspace"]["buffer"] = torch.empty((size(*sizes),), dtype=torch.uint8, device=DEVICE)
    return s["workspace"]["buffer"]


def plain_lora(s):
    at = s["adapter"].clamp(min=0).long()
    has = (s["adapter"] >= 0).float()[:, None]
    low = torch.bmm(s["a"][at].float(), s["x"].float()[:, :, None])              # [M, R, 1]
    add = torch.bmm(s["b"][at].float(), low)[:, :, 0]                            # [M, N]
    return s["base"] + add * (s["scale"][at][:, None] * has)


def plain_rope(s):
    Hq, Hkv, D, rot = s["Hq"], s["Hkv"], s["D"], s["rot"]
    M, pairs = s["qkv"].shape[0], rot // 2
    qkv = s["qkv"].reshape(M, Hq + 2 * Hkv, D)
    at = s["positions"].long()[s["axis"]].T                                     # [M, pairs]
    cs = s["table"][at, torch.arange(pairs, device=at.device)]                  # [M, pairs, 2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    qk = qkv[:, :Hq + Hkv]
    if s["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :pairs], qk[..., pairs:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    turned = torch.cat([turned, qk[..., rot:]], -1).to(s["q"].dtype)
    keep = s["slots"] >= 0
    to = s["slots"][keep]
    s["q"].copy_(turned[:, :Hq])
    s["k_cache"].view(-1, Hkv, D)[to] = turned[:, Hq:][keep]
    s["v_cache"].view(-1, Hkv, D)[to] = qkv[:, Hq + Hkv:][keep].to(s["q"].dtype)
    return s["q"], s["k_cache"], s["v_cache"]


def plain_attention(s):
    B, T, Hq, D = s["q"].shape
    Hkv, n = s["k_cache"].shape[2], s["prefix_len"]
    q = s["q"].float().reshape(B, T, Hkv, Hq // Hkv, D) * s["scale"]
    at = s["prefix_table"].long()
    kp = s["k_cache"][at].reshape(-1, Hkv, D)[:n].float()                       # [n, Hkv, D]
    vp = s["v_cache"][at].reshape(-1, Hkv, D)[:n].float()
    bt = s["own_table"].long()
    ko = s["k_cache"][bt].reshape(B, -1, Hkv, D)[:, :s["max_own"]].float()      # [B, max_own, Hkv, D]
    vo = s["v_cache"][bt].reshape(B, -1, Hkv, D)[:, :s["max_own"]].float()
    # token t of T sees the prefix and its request's own tokens up to itself
    last = s["own_len"][:, None] - T + torch.arange(T, device=q.device)          # [B, T]
    seen = torch.arange(s["max_own"], device=q.device) <= last[:, :, None]       # [B, T, max_own]
    sp = torch.einsum("bthgd,nhd->bthgn", q, kp)
    so = torch.einsum("bthgd,bnhd->bthgn", q, ko).masked_fill(~seen[:, :, None, None], -math.inf)
    top = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    sp, so = torch.exp(sp - top), torch.exp(so - top)
    total = sp.sum(-1) + so.sum(-1)
    o = torch.einsum("bthgn,nhd->bthgd", sp, vp) + torch.einsum("bthgn,bnhd->bthgd", so, vo)
    return (o / total[..., None]).reshape(B, T, Hq, D).to(s["q"].dtype)


def plain_logits(s):
    x, tok = s["logits"], s["tokens"].long()
    M, V = x.shape
    at = torch.arange(tok.shape[1], device=x.device)
    live = at < s["total_len"][:, None]
    answered = live & (at >= s["prompt_len"][:, None])
    count = torch.zeros((M, V), device=x.device).scatter_add_(1, tok, answered.float())
    seen = torch.zeros((M, V), device=x.device).scatter_add_(1, tok, live.float()) > 0
    rep = s["repetition"][:, None]
    y = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    y = y - (s["frequency"][:, None] * count + s["presence"][:, None] * (count > 0))
    if s["bias_tokens"] is not None:
        used = s["bias_tokens"] >= 0
        y = y.scatter_add(1, s["bias_tokens"].clamp(min=0).long(), s["bias_values"] * used)
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=x.device, dtype=torch.int32)) & 1
        allowed = bits.flatten(1)[:, :V].bool()[s["mask_row"].clamp(min=0).long()] | (s["mask_row"] < 0)[:, None]
        y = y.masked_fill(~allowed, -math.inf)
    return y


OWN = {"lora": own_lora, "rope": own_rope, "attention": own_attention, "logits": own_logits}
PLAIN = {"lora": plain_lora, "rope": plain_rope, "attention": plain_attention, "logits": plain_logits}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


def exact_lora(s):
    y = s["base"].double()
    for a in sorted(set(s["adapter"].tolist()) - {-1}):
        rows = (s["adapter"] == a).nonzero()[:, 0]
        low = s["x"][rows].double() @ s["a"][a].double().T
        y[rows] += s["scale"][a].double() * (low @ s["b"][a].double().T)
    return y


def exact_rope(s):
    Hq, Hkv, D, rot = s["Hq"], s["Hkv"], s["D"], s["rot"]
    M, pairs = s["qkv"].shape[0], rot // 2
    x = s["qkv"].double().reshape(M, -1, D).clone()
    for i in range(pairs):
        cs = s["table"][s["positions"][s["axis_of_pair"][i]].long(), i].double()
        turn = torch.complex(cs[:, 0], cs[:, 1])[:, None]
        lo, hi = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + pairs)
        z = torch.complex(x[:, :Hq + Hkv, lo], x[:, :Hq + Hkv, hi]) * turn
        x[:, :Hq + Hkv, lo], x[:, :Hq + Hkv, hi] = z.real, z.imag
    k, v = s["k_cache"].double().reshape(-1, Hkv, D), s["v_cache"].double().reshape(-1, Hkv, D)
    rows = (s["slots"] >= 0).nonzero()[:, 0]
    k[s["slots"][rows]], v[s["slots"][rows]] = x[rows, Hq:Hq + Hkv], x[rows, Hq + Hkv:]
    return x[:, :Hq], k.reshape(s["k_cache"].shape), v.reshape(s["v_cache"].shape)


def exact_attention(s):
    B, T, Hq, D = s["q"].shape
    Hkv, page, n = s["k_cache"].shape[2], s["k_cache"].shape[1], s["prefix_len"]
    G = Hq // Hkv
    y = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEVICE)
    first = s["prefix_table"].long()
    lens = s["own_len"].tolist()
    for h in range(Hkv):
        kp, vp = (c[first, :, h].reshape(-1, D)[:n].double() for c in (s["k_cache"], s["v_cache"]))
        for b in range(B):
            pages = s["own_table"][b, :(lens[b] + page - 1) // page].long()
            k, v = (torch.cat([p, c[pages, :, h].reshape(-1, D)[:lens[b]].double()])
                    for p, c in ((kp, s["k_cache"]), (vp, s["v_cache"])))
            z = s["q"][b, :, h * G:(h + 1) * G].reshape(T * G, D).double() @ k.T * s["scale"]
            for t in range(T - 1):
                z[t * G:(t + 1) * G, n + max(0, lens[b] - T + t + 1):] = -math.inf
            y[b, :, h * G:(h + 1) * G] = (torch.softmax(z, -1) @ v).reshape(T, G, D)
    return y


def exact_logits(s):
    y = s["logits"].double()
    M, V = y.shape
    for m in range(M):
        p, n = int(s["prompt_len"][m]), int(s["total_len"][m])
        once = torch.unique(s["tokens"][m, :n].long())
        r = s["repetition"][m].double()
        y[m, once] = torch.where(y[m, once] > 0, y[m, once] / r, y[m, once] * r)
        said, times = torch.unique(s["tokens"][m, p:n].long(), return_counts=True)
        y[m, said] -= s["frequency"][m].double() * times + s["presence"][m].double()
        if s["bias_tokens"] is not None:
            used = s["bias_tokens"][m] >= 0
            y[m, s["bias_tokens"][m][used].long()] += s["bias_values"][m][used].double()
        if s["mask"] is not None and int(s["mask_row"][m]) >= 0:
            at = torch.arange(V, device=DEVICE)
            word = s["mask"][int(s["mask_row"][m])][at // 32].long()
            y[m, ((word >> (at % 32)) & 1) == 0] = -math.inf
    return y


EXACT = {"lora": exact_lora, "rope": exact_rope, "attention": exact_attention, "logits": exact_logits}


# ---------------------------------------------------------------- what a pass cannot do without

def size(t):
    return 4 if t == "f32" else 2


def work(case):
    c = case
    if c["op"] == "lora":
        M, N, K, R = c["M"], c["N"], c["K"], c["R"]
        used = {"each": min(M, c["adapters"]), "shared": 1, "mixed": min(M, c["adapters"])}[c["spread"]]
        return {"bytes": M * K * size(c["x"]) + used * R * (K + N) * size(c["w"]) + 2 * M * N * 4,
                "flops": 2 * M * R * (K + N)}
    if c["op"] == "rope":
        M, out, turned = c["M"], (c["Hq"] + 2 * c["Hkv"]) * c["D"], (c["Hq"] + c["Hkv"]) * c["rot"]
        return {"bytes": M * out * (4 + 2) + min(M, c["positions"]) * c["rot"] * 4, "flops": 3 * M * turned}
    if c["op"] == "attention":
        B, T, Hq, Hkv, D = (c[k] for k in ("B", "T", "Hq", "Hkv", "D"))
        own_keys = c["own_max"] if B == 1 else B * (c["own_max"] + T) // 2
        return {"bytes": 2 * 2 * (c["prefix"] + own_keys) * Hkv * D + 2 * 2 * B * T * Hq * D,
                "flops": 4 * D * Hq * T * (B * c["prefix"] + own_keys)}
    M, V = c["M"], c["V"]
    return {"bytes": 2 * M * V * 4 + c["masks"] * V // 8 + M * (3 * c["history"] // 4) * 4 + M * c["biases"] * 8,
            "flops": M * V}
