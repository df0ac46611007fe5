"""The operators of a decode step over a cache held in 8 bits, and of the step's end.

- ``norm_rope``: RMS norms of each q and k head, rotary positions, append of k and v to a
  16-bit paged cache.
- ``append8``: the same, norms optional, into a cache of E4M3 codes with a power-of-two scale
  for each block of 16 tokens and head.
- ``attention8``: attention of each request's newest tokens over that cache.
- ``sample``: temperature, top-k, top-p and min-p, and a draw from given random numbers.

``listed`` names fixed cases, ``draw`` makes one of the same ranges, ``prepare`` makes a
case's inputs, ``run`` computes one pass (the plain form, or the library's calls where
``own`` is true), ``exact`` the same in 64 bits and ``work`` counts the bytes and operations
that a pass cannot do without.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
BLOCK = 16          # tokens that share a scale
EPS = 1e-6


# ---------------------------------------------------------------- cases

def norm_rope(name, M, Hq, Hkv, D, rot, axes, interleaved, type_, positions):
    return {"name": name, "op": "norm_rope", "M": M, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "axes": axes,
            "interleaved": interleaved, "type": type_, "positions": positions}


def append8(name, B, T, Hq, Hkv, D, rot, norms, interleaved, type_, before, page):
    """T tokens of each of B requests that have up to `before` tokens in the cache."""
    return {"name": name, "op": "append8", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "norms": norms,
            "interleaved": interleaved, "type": type_, "before": before, "page": page}


def attention8(name, B, T, Hq, Hkv, D, longest, page, type_):
    return {"name": name, "op": "attention8", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "longest": longest,
            "page": page, "type": type_}


def sample(name, M, V, spread, top_k, top_p, min_p, greedy):
    """spread: the logits' standard deviation; top_k, top_p, min_p: 0 for none, else what most
    rows have; greedy: some rows take the largest logit."""
    return {"name": name, "op": "sample", "M": M, "V": V, "spread": spread, "top_k": top_k, "top_p": top_p,
            "min_p": min_p, "greedy": greedy}


def listed():
    return [
        # one token of a decode step of an 8B-class model: latency counts
        norm_rope("norm_rope_one_token", 1, 32, 8, 128, 128, 1, False, "f16", 4096),
        # a prompt of 4001 tokens, 40 query heads over 8 key heads
        norm_rope("norm_rope_prompt", 4001, 40, 8, 128, 128, 1, False, "bf16", 32768),
        # a decode step of 64 requests, a token each, into blocks that are partly full
        append8("append8_batch", 64, 1, 32, 8, 128, 128, True, False, "f16", 2000, 64),
        # prompts of 3 requests, 1335 tokens each
        append8("append8_prompt", 3, 1335, 40, 8, 128, 128, False, False, "bf16", 100, 64),
        # one request of a few hundred tokens: latency counts
        attention8("attention8_one_request", 1, 1, 32, 8, 128, 560, 16, "f16"),
        # an ordinary batch
        attention8("attention8_batch", 24, 1, 40, 8, 128, 8191, 64, "bf16"),
        # speculative verification: 5 tokens of each request, 64-wide heads
        attention8("attention8_verify", 16, 5, 32, 4, 64, 4099, 32, "f16"),
        # one request with a very long document
        attention8("attention8_long_document", 1, 1, 40, 8, 128, 131072, 64, "bf16"),
        # a full batch of long conversations
        attention8("attention8_full_batch", 64, 1, 40, 8, 128, 16384, 64, "f16"),
        # one row of a small vocabulary: latency counts
        sample("sample_one_row", 1, 32000, 3.0, 40, 0.95, 0.0, False),
        # eight rows of a large vocabulary, by probability mass alone
        sample("sample_eight_rows", 8, 151936, 4.0, 0, 0.9, 0.05, False),
        # a full batch, each row with its own settings
        sample("sample_full_batch", 96, 151936, 4.0, 50, 0.95, 0.02, True),
    ]


def spread_over(rng, low, high):
    """A whole number of low..high, even over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append8", "attention8", "sample"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.randint(1, 8)
    type_ = rng.choice(["f16", "bf16"])
    if op == "norm_rope":
        D = rng.choice([64, 80, 128, 256])
        M = spread_over(rng, 1, 4001)
        while M * (Hq + 2 * Hkv) * D > 4001 * 56 * 128:
            M //= 2
        c = norm_rope("", M, Hq, Hkv, D, rng.choice([D, D, D // 2]), rng.choice([1, 3]), rng.random() < 0.4, type_,
                      spread_over(rng, 4096, 65536))
    elif op == "append8":
        D = rng.choice([64, 128, 128])
        B, T = spread_over(rng, 1, 96), rng.choice([1, 1, 2, 5, 8, 16, 77, 300, 1335])
        while B * T > 4005:
            B = max(1, B // 2)
        c = append8("", B, T, Hq, Hkv, D, rng.choice([D, D, D // 2]), rng.random() < 0.6, rng.random() < 0.3, type_,
                    spread_over(rng, 1, 4000), rng.choice([16, 32, 64, 128]))
    elif op == "attention8":
        B, T, D = spread_over(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8]), rng.choice([64, 128, 128])
        longest = max(T, spread_over(rng, 1, 131072))
        while B * longest * Hkv * D > 64 * 16384 * 8 * 128 or B * T * longest * Hq > 64 * 16384 * 40:
            longest //= 2
        c = attention8("", B, T, Hq, Hkv, D, max(T, longest), rng.choice([16, 32, 64, 128]), type_)
    else:
        c = sample("", spread_over(rng, 1, 96), spread_over(rng, 1000, 151936), rng.choice([0.5, 2.0, 4.0, 8.0]),
                   rng.choice([0, 1, 20, 50, 1000]), rng.choice([0.0, 0.5, 0.9, 0.99]), rng.choice([0.0, 0.0, 0.05, 0.3]),
                   rng.random() < 0.3)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 7919 + 23)
    return {"norm_rope": prepare_norm_rope, "append8": prepare_append8, "attention8": prepare_attention8,
            "sample": prepare_sample}[case["op"]](case, g)


def normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * scale).to(dtype)


def whole(g, low, high, shape, dtype=torch.int32):
    return torch.randint(low, high, shape, generator=g, device=DEVICE, dtype=dtype)


def angles(positions, pairs):
    inv = 1e6 ** -(torch.arange(pairs, dtype=torch.float64, device=DEVICE) / pairs)
    angle = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * inv
    return torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32).contiguous()


def head_norm(g, D):
    return normal(g, (D,), scale=0.2) + 1.0


def prepare_norm_rope(c, g):
    M, Hq, Hkv, D, rot, A = (c[k] for k in ("M", "Hq", "Hkv", "D", "rot", "axes"))
    pairs, dtype, page = rot // 2, TYPES[c["type"]], 16
    pages = (2 * M + 64 + page - 1) // page
    slots = torch.randperm(pages * page, generator=g, device=DEVICE)[:M].to(torch.int64)   # free places, in no order
    axis = [i * A // pairs for i in range(pairs)]
    return {"op": "norm_rope", "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "interleaved": c["interleaved"],
            "axis_of_pair": bytes(axis), "axis": torch.tensor(axis, device=DEVICE),
            "qkv": normal(g, (M, (Hq + 2 * Hkv) * D), scale=2.0),       # the shared projection's output
            "positions": whole(g, 0, c["positions"], (A, M)), "table": angles(c["positions"], pairs), "slots": slots,
            "q_norm": head_norm(g, D), "k_norm": head_norm(g, D),
            "k_cache": normal(g, (pages, page, Hkv, D), dtype), "v_cache": normal(g, (pages, page, Hkv, D), dtype),
            "q": torch.empty((M, Hq, D), dtype=dtype, device=DEVICE)}


def codes(g, pages, page, Hkv, D):
    """Codes as an append leaves them, the largest of a block near 448, and scales of blocks and heads."""
    x = torch.randn((pages, page, Hkv, D), generator=g, device=DEVICE, dtype=torch.float16) * 110.0
    scale = torch.exp2(whole(g, -8, -5, (pages, page // BLOCK, Hkv)).float())
    return x.clamp(-448.0, 448.0).to(E4M3), scale


def prepare_append8(c, g):
    B, T, Hq, Hkv, D, rot, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "rot", "page"))
    M, pairs, width = B * T, rot // 2, (c["before"] + T + page - 1) // page
    had = whole(g, 0, c["before"] + 1, (B,), torch.int64)
    table = torch.randperm(B * width + 2, generator=g, device=DEVICE)[:B * width].reshape(B, width)
    at = had[:, None] + torch.arange(T, device=DEVICE)                          # [B, T] the tokens' positions
    slots = (table.gather(1, at // page) * page + at % page).reshape(M)
    padding = M // 16 if T == 1 else 0                                          # a batch that is not full
    if padding:
        slots[M - padding:] = -1
    k_cache, k_scale = codes(g, B * width + 2, page, Hkv, D)
    v_cache, v_scale = codes(g, B * width + 2, page, Hkv, D)
    return {"op": "append8", "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "interleaved": c["interleaved"],
            "axis_of_pair": bytes(pairs), "axis": torch.zeros((pairs,), dtype=torch.int64, device=DEVICE),
            "qkv": normal(g, (M, (Hq + 2 * Hkv) * D), scale=1.5),
            "positions": at.reshape(1, M).to(torch.int32), "table": angles(c["before"] + T, pairs), "slots": slots,
            "q_norm": head_norm(g, D) if c["norms"] else None, "k_norm": head_norm(g, D) if c["norms"] else None,
            "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale,
            "q": torch.empty((M, Hq, D), dtype=TYPES[c["type"]], device=DEVICE)}


def prepare_attention8(c, g):
    B, T, Hq, Hkv, D, longest, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "longest", "page"))
    width = (longest + page - 1) // page
    lens = whole(g, T, longest + 1, (B,))
    lens[0] = longest
    k_cache, k_scale = codes(g, B * width + 3, page, Hkv, D)
    v_cache, v_scale = codes(g, B * width + 3, page, Hkv, D)
    table = torch.randperm(B * width + 3, generator=g, device=DEVICE)[:B * width].to(torch.int32)   # in no order
    return {"op": "attention8", "max_len": longest, "scale": 1 / math.sqrt(D),
            "q": normal(g, (B, T, Hq, D), TYPES[c["type"]], 1.2),
            "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale,
            "table": table.reshape(B, width).contiguous(), "lens": lens,
            "out": torch.empty((B, T, Hq, D), dtype=TYPES[c["type"]], device=DEVICE), "workspace": {}}


def prepare_sample(c, g):
    M, V = c["M"], c["V"]
    most = torch.rand((M,), generator=g, device=DEVICE) < 0.8                   # the other rows have none
    temperature = torch.rand((M,), generator=g, device=DEVICE) * 0.9 + 0.4
    if c["greedy"]:
        temperature = torch.where(torch.rand((M,), generator=g, device=DEVICE) < 0.15, 0.0, temperature)
    return {"op": "sample", "logits": normal(g, (M, V), scale=c["spread"]),
            "u": torch.rand((M,), generator=g, device=DEVICE), "temperature": temperature,
            "top_k": torch.where(most, c["top_k"], 0).to(torch.int32) if c["top_k"] else None,
            "top_p": torch.where(most.roll(1), c["top_p"], 1.0) if c["top_p"] else None,
            "min_p": torch.where(most.roll(2), c["min_p"], 0.0) if c["min_p"] else None,
            "token": torch.empty((M,), dtype=torch.int32, device=DEVICE),
            "prob": torch.empty((M,), dtype=torch.float32, device=DEVICE)}


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return OWN[state["op"]](state)
    return PLAIN[state["op"]](state)


def own_norm_rope(s):
    import gemm_qmv_quantize_gb300 as q
    q.qmv_norm_rope_append(s["qkv"], s["positions"], s["table"], s["axis_of_pair"], s["slots"], s["k_cache"],
                           s["v_cache"], s["q_norm"], s["k_norm"], eps=EPS, interleaved=s["interleaved"], out=s["q"])
    return s["q"], s["k_cache"], s["v_cache"]


def own_append8(s):
    import gemm_qmv_quantize_gb300 as q
    q.qmv_rope_append_e4m3(s["qkv"], s["positions"], s["table"], s["axis_of_pair"], s["slots"], s["k_cache"],
                           s["v_cache"], s["k_scale"], s["v_scale"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                           interleaved=s["interleaved"], out=s["q"])
    return s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def own_attention8(s):
    import gemm_qmv_quantize_gb300 as q
    if "buffer" not in s["workspace"]:      # which a user's program keeps for calls of these sizes
        need = q.qmv_paged_attention_e4m3_workspace(*s["q"].shape[:3], s["k_cache"].shape[2], s["q"].shape[3], s["max_len"])
        s["workspace"]["buffer"] = torch.empty((need,), dtype=torch.uint8, device=DEVICE)
    return q.qmv_paged_attention_e4m3(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                      s["lens"], scale=s["scale"], max_len=s["max_len"], out=s["out"],
                                      workspace=s["workspace"]["buffer"])


def own_sample(s):
    import gemm_qmv_quantize_gb300 as q
    q.qmv_sample(s["logits"], s["u"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                 out=s["token"], prob=s["prob"])
    return s["token"], s["prob"]


def normed(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def turned(s):
    """q, k (normed and turned) and v heads in fp32, [M, H, D]."""
    Hq, Hkv, D, rot = s["Hq"], s["Hkv"], s["D"], s["rot"]
    M, pairs = s["qkv"].shape[0], rot // 2
    x = s["qkv"].reshape(M, Hq + 2 * Hkv, D)
    qk = torch.cat([normed(x[:, :Hq], s["q_norm"]), normed(x[:, Hq:Hq + Hkv], s["k_norm"])], 1)
    at = s["positions"].long()[s["axis"]].T                                     # [M, pairs]
    cs = s["table"][at, torch.arange(pairs, device=at.device)]                  # [M, pairs, 2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if s["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        first = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :pairs], qk[..., pairs:rot]
        first = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([first, qk[..., rot:]], -1)
    return qk[:, :Hq], qk[:, Hq:], x[:, Hq + Hkv:]


def plain_norm_rope(s):
    q, k, v = turned(s)
    keep = s["slots"] >= 0
    to = s["slots"][keep]
    s["q"].copy_(q)
    s["k_cache"].view(-1, s["Hkv"], s["D"])[to] = k[keep].to(s["q"].dtype)
    s["v_cache"].view(-1, s["Hkv"], s["D"])[to] = v[keep].to(s["q"].dtype)
    return s["q"], s["k_cache"], s["v_cache"]


def scale_for(largest):
    """The least power of two (2^-64 at least) of which 448 is not below `largest`."""
    m, e = torch.frexp(largest)                                                 # largest = m 2^e, 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(largest), torch.where(largest > 0, e, -64).clamp(min=-64))


def put8(x, slots, cache, scales):
    """x fp32 [n, Hkv, D] to its slots: the blocks' scales grow where they have to, and the codes that a
    block had before the first of the new ones follow."""
    Hkv, D = x.shape[1:]
    blocks = scales.numel() // Hkv
    block, offset = slots // BLOCK, slots % BLOCK
    largest = torch.zeros((blocks, Hkv), device=x.device).index_reduce_(0, block, x.abs().amax(-1), "amax")
    first = torch.full((blocks,), BLOCK, device=x.device).index_reduce_(0, block, offset, "amin")
    touched = torch.unique(block)
    need, had = scale_for(largest[touched]), scales.view(blocks, Hkv)[touched]
    scale = torch.where((first[touched] > 0)[:, None], torch.maximum(had, need), need)
    old = cache.view(blocks, BLOCK, Hkv, D)[touched]
    moved = (old.float() * (had / scale)[:, None, :, None]).to(E4M3)
    kept = torch.arange(BLOCK, device=x.device) < first[touched][:, None]
    bytes_ = cache.view(torch.uint8).view(blocks, BLOCK, Hkv, D)
    bytes_[touched] = torch.where(kept[:, :, None, None], moved.view(torch.uint8), old.view(torch.uint8))
    scales.view(blocks, Hkv)[touched] = scale
    bytes_.view(-1, Hkv, D)[slots] = (x / scales.view(blocks, Hkv)[block][:, :, None]).to(E4M3).view(torch.uint8)


def plain_append8(s):
    q, k, v = turned(s)
    s["q"].copy_(q)
    keep = s["slots"] >= 0
    to = s["slots"][keep]
    put8(k[keep], to, s["k_cache"], s["k_scale"])
    put8(v[keep], to, s["v_cache"], s["v_scale"])
    return s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def gathered(s, cache, scale):
    """The requests' keys or values in fp32, [B, max_len, Hkv, D]."""
    at = s["table"].long()
    B, Hkv, D = at.shape[0], cache.shape[2], cache.shape[3]
    x = cache.view(torch.uint8)[at].view(E4M3).float().reshape(B, -1, BLOCK, Hkv, D)
    x *= scale[at].reshape(B, -1, 1, Hkv, 1)
    return x.reshape(B, -1, Hkv, D)[:, :s["max_len"]]


def plain_attention8(s):
    B, T, Hq, D = s["q"].shape
    Hkv, n = s["k_cache"].shape[2], s["max_len"]
    q = s["q"].float().reshape(B, T, Hkv, Hq // Hkv, D) * s["scale"]
    # token t of T sees its request's tokens up to itself
    last = s["lens"][:, None] - T + torch.arange(T, device=q.device)             # [B, T]
    seen = torch.arange(n, device=q.device) <= last[:, :, None]                  # [B, T, n]
    z = torch.einsum("bthgd,bnhd->bthgn", q, gathered(s, s["k_cache"], s["k_scale"]))
    z = z.masked_fill(~seen[:, :, None, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    o = torch.einsum("bthgn,bnhd->bthgd", p, gathered(s, s["v_cache"], s["v_scale"]))
    return (o / p.sum(-1, keepdim=True)).reshape(B, T, Hq, D).to(s["q"].dtype)


def plain_sample(s):
    x = s["logits"]
    M, V = x.shape
    order = torch.sort(x, dim=1, descending=True, stable=True)                  # ties: the lowest index first
    top, rank = order.values[:, :1].double(), torch.arange(V, device=x.device)
    greedy = s["temperature"] <= 0
    temperature = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"]).double()[:, None]
    w = torch.exp((order.values.double() - top) / temperature)
    keep = torch.ones((M, V), dtype=torch.bool, device=x.device)
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
        keep &= rank < k
    if s["top_p"] is not None:
        among = torch.where(keep, w, 0.0)
        upto = torch.cumsum(among, 1)
        keep &= (upto - among < s["top_p"].double()[:, None] * upto[:, -1:]) | (s["top_p"][:, None] >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    keep &= ~greedy[:, None]
    keep[:, 0] = True
    by_index = torch.zeros((M, V), dtype=torch.float64, device=x.device).scatter_(1, order.indices, torch.where(keep, w, 0.0))
    upto = torch.cumsum(by_index, 1)
    token = (upto <= s["u"].double()[:, None] * upto[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
    prob = by_index.gather(1, token) / upto[:, -1:]
    return token[:, 0].to(torch.int32), prob[:, 0].to(torch.float32)


OWN = {"norm_rope": own_norm_rope, "append8": own_append8, "attention8": own_attention8, "sample": own_sample}
PLAIN = {"norm_rope": plain_norm_rope, "append8": plain_append8, "attention8": plain_attention8, "sample": plain_sample}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


def exact_heads(s):
    """All heads in 64 bits after norm and turn."""
    Hq, Hkv, D, rot = s["Hq"], s["Hkv"], s["D"], s["rot"]
    x = s["qkv"].double().reshape(-1, Hq + 2 * Hkv, D).clone()
    for weight, heads in ((s["q_norm"], slice(0, Hq)), (s["k_norm"], slice(Hq, Hq + Hkv))):
        if weight is not None:
            rms = torch.linalg.vector_norm(x[:, heads], dim=-1, keepdim=True) ** 2 / D + EPS
            x[:, heads] = x[:, heads] / rms.sqrt() * weight.double()
    for i in range(rot // 2):
        cs = s["table"][s["positions"][s["axis_of_pair"][i]].long(), i].double()
        lo, hi = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + rot // 2)
        z = torch.complex(x[:, :Hq + Hkv, lo], x[:, :Hq + Hkv, hi]) * torch.complex(cs[:, 0], cs[:, 1])[:, None]
        x[:, :Hq + Hkv, lo], x[:, :Hq + Hkv, hi] = z.real, z.imag
    return x


def exact_norm_rope(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    x = exact_heads(s)
    k, v = s["k_cache"].double().reshape(-1, Hkv, D), s["v_cache"].double().reshape(-1, Hkv, D)
    k[s["slots"]], v[s["slots"]] = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return x[:, :Hq], k.reshape(s["k_cache"].shape), v.reshape(s["v_cache"].shape)


def to_e4m3(x):
    """Rounded to the nearest value of 4 significant bits and a least exponent of -6, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact_append8(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    x = exact_heads(s)
    made = [x[:, :Hq]]
    slots = s["slots"].tolist()
    by_block = {}
    for m, slot in enumerate(slots):
        if slot >= 0:
            by_block.setdefault(slot // BLOCK, []).append(m)
    scales = []
    for which, (name, heads) in enumerate((("k", slice(Hq, Hq + Hkv)), ("v", slice(Hq + Hkv, Hq + 2 * Hkv)))):
        cache = s[name + "_cache"].double().reshape(-1, Hkv, D)
        scale = s[name + "_scale"].double().reshape(-1, Hkv)
        for block, rows in by_block.items():
            new = x[rows, heads]                                                # [n, Hkv, D]
            need = torch.exp2(torch.ceil(torch.log2(new.abs().amax((0, 2)) / 448)).clamp(min=-64))
            first = min(slots[m] % BLOCK for m in rows)
            if first:
                need = torch.maximum(need, scale[block])
                kept = cache[block * BLOCK:block * BLOCK + first]
                cache[block * BLOCK:block * BLOCK + first] = to_e4m3(kept * (scale[block] / need)[None, :, None])
            scale[block] = need
            cache[[slots[m] for m in rows]] = to_e4m3(new / need[None, :, None])
        made.append(cache.reshape(s[name + "_cache"].shape))
        scales.append(scale.reshape(s[name + "_scale"].shape))
    return (*made, *scales)


def exact_attention8(s):
    B, T, Hq, D = s["q"].shape
    Hkv, page = s["k_cache"].shape[2], s["k_cache"].shape[1]
    G = Hq // Hkv
    y = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :(n + page - 1) // page].long()
        for h in range(Hkv):
            k, v = (c.view(torch.uint8)[pages, :, h].view(E4M3).double().reshape(-1, BLOCK, D)
                    * z[pages, :, h].double().reshape(-1, 1, 1)
                    for c, z in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            k, v = k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]
            z = s["q"][b, :, h * G:(h + 1) * G].reshape(T * G, D).double() @ k.T * s["scale"]
            for t in range(T - 1):
                z[t * G:(t + 1) * G, n - T + t + 1:] = -math.inf
            y[b, :, h * G:(h + 1) * G] = (torch.softmax(z, -1) @ v).reshape(T, G, D)
    return y


def exact_sample(s):
    """The probability of the token that the row's random number falls to."""
    M, V = s["logits"].shape
    made = torch.zeros((M,), dtype=torch.float64, device=DEVICE)
    for m in range(M):
        x, T = s["logits"][m].double(), float(s["temperature"][m])
        ids = torch.argsort(x, descending=True, stable=True)
        if T <= 0:
            ids = ids[:1]
        if s["top_k"] is not None and int(s["top_k"][m]) > 0:
            ids = ids[:int(s["top_k"][m])]
        p = torch.softmax(x[ids] / (T if T > 0 else 1.0), 0)
        n = len(ids)
        if s["top_p"] is not None and float(s["top_p"][m]) < 1:
            n = max(1, int((torch.cumsum(p, 0) - p < float(s["top_p"][m])).sum()))
        if s["min_p"] is not None:
            n = max(1, min(n, int((p >= float(s["min_p"][m]) * p[0]).sum())))
        ids, p = ids[:n], p[:n] / p[:n].sum()
        ids, at = torch.sort(ids)
        p = p[at]
        made[m] = p[min(int((torch.cumsum(p, 0) <= float(s["u"][m])).sum()), n - 1)]
    return None, made


EXACT = {"norm_rope": exact_norm_rope, "append8": exact_append8, "attention8": exact_attention8, "sample": exact_sample}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "norm_rope":
        M, out, qk = c["M"], (c["Hq"] + 2 * c["Hkv"]) * c["D"], (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": M * out * (4 + 2) + min(M, c["positions"]) * c["rot"] * 4, "flops": 7 * M * qk}
    if c["op"] == "append8":
        M, kv = c["B"] * c["T"], 2 * c["Hkv"] * c["D"]
        return {"bytes": M * ((c["Hq"] * c["D"] + kv) * 4 + c["Hq"] * c["D"] * 2 + kv + c["rot"] * 4)
                + 2 * 2 * c["Hkv"] * 4 * (M // BLOCK + c["B"]), "flops": 7 * M * (c["Hq"] * c["D"] + kv)}
    if c["op"] == "attention8":
        B, T, Hq, Hkv, D = (c[k] for k in ("B", "T", "Hq", "Hkv", "D"))
        keys = c["longest"] if B == 1 else c["longest"] + (B - 1) * (c["longest"] + T) // 2
        return {"bytes": 2 * keys * Hkv * D + 2 * 4 * Hkv * (keys // BLOCK) + 2 * 2 * B * T * Hq * D,
                "flops": 4 * D * Hq * T * keys}
    return {"bytes": 4 * c["M"] * c["V"] + 32 * c["M"], "flops": 4 * c["M"] * c["V"]}
