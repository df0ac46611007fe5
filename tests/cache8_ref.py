"""Plain definitions in 64 bits of the operators over a cache of E4M3 codes, of the norms of
q and k, and of sampling, for the GPU tests; and inputs that several tests share."""
import math

import torch

import decode_ref

E4M3 = torch.float8_e4m3fn


def normed(x, weight, eps):
    """x [..., D] over its root mean square, times the weight, in 64 bits."""
    x = x.double()
    return x if weight is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def heads(qkv, positions, table, axis_of_pair, Hkv, D, interleaved, q_norm, k_norm, eps):
    """q, k, v heads [M, H, D] in 64 bits after norm and turn."""
    x = qkv.double().reshape(qkv.shape[0], qkv.shape[1] // D, D).clone()
    Hq = x.shape[1] - 2 * Hkv
    x[:, :Hq] = normed(x[:, :Hq], q_norm, eps)
    x[:, Hq:Hq + Hkv] = normed(x[:, Hq:Hq + Hkv], k_norm, eps)
    return decode_ref.rope(x.reshape(qkv.shape[0], -1), positions, table, axis_of_pair, Hkv, D, interleaved)


def scale_for(largest):
    """The least power of two, 2^-64 at least, of which 448 is not below `largest` (a float)."""
    if largest == 0:
        return 2.0 ** -64
    m, e = math.frexp(largest)
    return 2.0 ** max(-64, e - 9 if m <= 0.875 else e - 8)


def append(x, slots, cache, scale):
    """The new values x (64 bits, [M, Hkv, D]) into copies of codes and scales: (codes as 64-bit
    values, scales, the new values that each slot's codes stand for, with NaN elsewhere)."""
    Hkv, D = cache.shape[2:]
    codes, scale = cache.double().reshape(-1, Hkv, D).clone(), scale.double().reshape(-1, Hkv).clone()
    wanted = torch.full_like(codes, math.nan)
    runs = {}
    for m, s in enumerate(slots.tolist()):
        if 0 <= s < codes.shape[0]:
            runs.setdefault(s // 16, []).append((m, s))
    for block, rows in runs.items():
        first = rows[0][1] % 16
        for h in range(Hkv):
            new = x[[m for m, _ in rows], h]
            fine = new[torch.isfinite(new)]
            s = scale_for(float(fine.abs().max()) if fine.numel() else 0.0)
            if first:
                had = float(scale[block, h])
                s = max(s, had)
                kept = codes[block * 16:block * 16 + first, h]
                codes[block * 16:block * 16 + first, h] = (kept * (had / s)).float().to(E4M3).double()
            scale[block, h] = s
        for m, s in rows:
            wanted[s] = torch.where(torch.isinf(x[m]), math.nan, x[m])
            codes[s] = math.nan
    return codes, scale, wanted


def values(cache, scale):
    """The values [pages, page, Hkv, D] that codes stand for."""
    pages, page, Hkv, D = cache.shape
    return (cache.double().reshape(pages, page // 16, 16, Hkv, D) * scale.double()[:, :, None, :, None]).reshape(cache.shape)


def attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale):
    """(o, bound, floor): bound = sum_j p_j |V_j|; floor = max_j (p_j sv_j) sum_j |code_j|, to which the terms
    below binary16's normal range are rounded."""
    B, T, Hq, D = q.shape
    page, Hkv = k_cache.shape[1:3]
    G = Hq // Hkv
    o = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=q.device)
    bound, floor = torch.zeros_like(o), torch.zeros_like(o)
    for b in range(B):
        total = max(0, int(lens[b]))
        at = table[b, :(total + page - 1) // page].long()
        pick = lambda c: c.view(torch.uint8)[at].view(E4M3)  # noqa: E731
        k = values(pick(k_cache), k_scale[at]).reshape(-1, Hkv, D)
        v = values(pick(v_cache), v_scale[at]).reshape(-1, Hkv, D)
        codes = pick(v_cache).double().reshape(-1, Hkv, D)
        sv = v_scale[at].double().repeat_interleave(16, 1).reshape(-1, Hkv)
        for t in range(T):
            n = max(0, total - T + 1 + t)
            if n == 0:
                continue
            for h in range(Hq):
                j = h // G
                p = torch.softmax(k[:n, j] @ q[b, t, h].double() * scale, 0)
                o[b, t, h], bound[b, t, h] = p @ v[:n, j], p @ v[:n, j].abs()
                floor[b, t, h] = (p * sv[:n, j]).max() * codes[:n, j].abs().sum(0)
    return o, bound, floor


def random_cache(g, pages, page, Hkv, D, low=-9, high=-4):
    x = torch.randn((pages, page, Hkv, D), generator=g, device="cuda") * 100
    s = torch.exp2(torch.randint(low, high, (pages, page // 16, Hkv), generator=g, device="cuda").float())
    return x.clamp(-448, 448).to(E4M3), s


def kept(x, temperature, top_k, top_p, min_p):
    """(indices of the kept tokens in ascending order, their weights) of a row, in 64 bits."""
    x = torch.where(torch.isnan(x), -math.inf, x.double())
    order = torch.argsort(x, descending=True, stable=True)
    top = x[order[0]]
    if top == -math.inf:
        return order[:0], x[:0]
    w = torch.ones_like(x) if top == math.inf else torch.exp((x - top) / (temperature if temperature > 0 else 1.0))
    w = torch.where(x == -math.inf, 0.0, torch.where(x == math.inf, 1.0, w if top < math.inf else 0.0))[order]
    n = len(w)
    if 0 < top_k < n:
        n = top_k
    if top_p < 1:
        upto = torch.cumsum(w[:n], 0)
        n = int((upto - w[:n] < top_p * upto[-1]).sum())
    if min_p > 0:
        n = min(n, int((w >= min_p).sum()))
    if not temperature > 0:
        n = 1
    ids, at = torch.sort(order[:max(1, n)])
    return ids, w[:max(1, n)][at]
