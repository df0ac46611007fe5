"""Plain definitions in 64 bits of the operators beside the matmuls, for the GPU tests.

Each returns the value and, where the operator sums, a bound to which the tests' derived
tolerances are relative (the same sum over absolute values).
"""
import math

import torch


def lora(x, a, b, adapter, scale, base):
    """(y, bound): bound[m][n] = |scale| sum_r |B| sum_k |A x|."""
    y, bound = base.double().clone(), torch.zeros_like(base, dtype=torch.float64)
    for m, l in enumerate(adapter.tolist()):
        if 0 <= l < a.shape[0]:
            xd, ad, bd, s = x[m].double(), a[l].double(), b[l].double(), scale[l].double()
            y[m] += s * (bd @ (ad @ xd))
            bound[m] = s.abs() * (bd.abs() @ (ad.abs() @ xd.abs()))
    return y, bound


def rope(qkv, positions, table, axis_of_pair, Hkv, D, interleaved):
    """q, k, v heads [M][H][D] after the turn."""
    M, pairs = qkv.shape[0], table.shape[1]
    x = qkv.double().reshape(M, -1, D).clone()
    turned = x.shape[1] - Hkv
    for i in range(pairs):
        cs = table[positions[axis_of_pair[i]].long(), i].double()
        c, s = cs[:, :1], cs[:, 1:]
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        u, v = x[:, :turned, lo].clone(), x[:, :turned, hi].clone()
        x[:, :turned, lo], x[:, :turned, hi] = u * c - v * s, v * c + u * s
    return x[:, :turned - Hkv], x[:, turned - Hkv:turned], x[:, turned:]


def keys_of(cache, table, n):
    """The first n rows [n][Hkv][D] of the pages that `table` lists."""
    page = cache.shape[1]
    return cache[table[:(n + page - 1) // page].long()].reshape(-1, *cache.shape[2:])[:n].double()


def attention(q, k_cache, v_cache, prefix_table, prefix_len, own_table, own_len, scale):
    """(o, bound): bound = sum_j p_j |V_j|."""
    B, T, Hq, D = q.shape
    G = Hq // k_cache.shape[2]
    o = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    kp, vp = (keys_of(c, prefix_table, prefix_len) for c in (k_cache, v_cache))
    for b in range(B):
        for t in range(T):
            n = max(0, int(own_len[b]) - T + 1 + t)
            k, v = (torch.cat([p, keys_of(c, own_table[b], n)]) for p, c in ((kp, k_cache), (vp, v_cache)))
            if k.shape[0] == 0:
                continue
            for h in range(Hq):
                p = torch.softmax(k[:, h // G] @ q[b, t, h].double() * scale, 0)
                o[b, t, h], bound[b, t, h] = p @ v[:, h // G], p @ v[:, h // G].abs()
    return o, bound


def logits(x, tokens, prompt_len, total_len, repetition, presence, frequency, bias_tokens, bias_values, mask, mask_row):
    y = x.double().cpu().clone()
    M, V = y.shape
    for m in range(M):
        n = min(int(total_len[m]), tokens.shape[1])
        history = tokens[m, :n].tolist()
        once = {t for t in history if 0 <= t < V}
        answered = {}
        for t in history[max(0, int(prompt_len[m])):]:
            if 0 <= t < V:
                answered[t] = answered.get(t, 0) + 1
        for t in once:
            r = 1.0 if repetition is None else float(repetition[m])
            y[m, t] = y[m, t] / r if y[m, t] > 0 else y[m, t] * r
        for t, c in answered.items():
            y[m, t] -= (0.0 if frequency is None else float(frequency[m])) * c
            y[m, t] -= 0.0 if presence is None else float(presence[m])
        if bias_tokens is not None:
            for t, v in zip(bias_tokens[m].tolist(), bias_values[m].tolist()):
                if 0 <= t < V:
                    y[m, t] += v
        row = m if mask_row is None else int(mask_row[m])
        if mask is not None and 0 <= row < mask.shape[0]:
            words = mask[row].cpu().numpy().view("uint32")
            for v in range(V):
                if not (int(words[v // 32]) >> (v % 32)) & 1:
                    y[m, v] = -math.inf
    return y
