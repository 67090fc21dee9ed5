"""Plain 64-bit forms of the paged serving operators, request by request, and the error bounds of their outputs."""
from __future__ import annotations

import numpy as np
import torch


def plan(cached, new, page, max_pages, num_pages, max_tokens, table, free, count):
    """(dict of outputs, refused) of a page plan on host lists and numpy arrays; the arrays are copied."""
    table, free = table.copy(), free.copy()
    need = [-(-(c + n) // page) - -(-c // page) if n >= 0 else 0 for c, n in zip(cached, new)]
    back = [-(-c // page) if n < 0 else 0 for c, n in zip(cached, new)]
    bad = (any(c < 0 or c + max(n, 0) > max_pages * page for c, n in zip(cached, new))
           or sum(max(n, 0) for n in new) > max_tokens or not 0 <= count <= num_pages or sum(need) > count
           or count - sum(need) + sum(back) > num_pages)
    pos, slot = np.zeros(max_tokens, np.int32), np.full(max_tokens, -1, np.int32)
    if bad:
        return {"table": table, "free": free, "count": count, "cu": np.zeros(len(new) + 1, np.int32),
                "kv": np.array(cached, np.int32), "pos": pos, "slot": slot}, True
    top, t, cu = count, 0, [0]
    for b, (c, n) in enumerate(zip(cached, new)):
        for k in range(-(-c // page), -(-c // page) + need[b]):
            top -= 1
            table[b, k] = free[top]
        for p in range(c, c + max(n, 0)):
            pos[t] = p
            g = table[b, p // page]
            slot[t] = g * page + p % page if 0 <= g < num_pages else -1
            t += 1
        cu.append(t)
    for b, n in enumerate(new):
        for k in range(back[b]):
            free[top] = table[b, k] if 0 <= table[b, k] < num_pages else -1
            top += 1
    kv = [0 if n < 0 and c > 0 else c + max(n, 0) for c, n in zip(cached, new)]
    return {"table": table, "free": free, "count": top, "cu": np.array(cu, np.int32), "kv": np.array(kv, np.int32),
            "pos": pos, "slot": slot}, False


def gather(pages, table_row, n):
    """The first n rows [n][kv heads][D] that a block-table row lists, in 64 bits (pages outside the pool are zero)."""
    P, Hkv, ps, D = pages.shape
    ids = torch.as_tensor(table_row[: -(-n // ps)], device=pages.device).long()
    ok = (ids >= 0) & (ids < P)
    x = pages[ids.clamp(0, P - 1)].double()
    x[~ok] = 0.0
    return x.transpose(1, 2).reshape(-1, Hkv, D)[:n]


def attention(q, k, v):
    """q [n][H][D] at the last n of len(k) positions: (out, bound weights) in 64 bits.

    Returns out [n][H][D], A = sum_j p_j |v_j| and E = max_j sum_d |q_d k_jd| / sqrt(D) over the visible keys."""
    n, H, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, A, E = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(n, H, 1, dtype=torch.float64, device=q.device)
    for i in range(n):
        p = L - n + i
        if p < 0:
            continue
        ks, vs = k[: p + 1], v[: p + 1]
        for g in range(Hkv):
            r = H // Hkv
            qq = q[i, g * r:(g + 1) * r]
            s = qq @ ks[:, g].T / D ** 0.5
            w = torch.softmax(s, -1)
            out[i, g * r:(g + 1) * r] = w @ vs[:, g]
            A[i, g * r:(g + 1) * r] = w @ vs[:, g].abs()
            E[i, g * r:(g + 1) * r, 0] = (qq.abs() @ ks[:, g].abs().T / D ** 0.5).amax(-1)
    return out, A, E


def attention_bound(out, A, E, keys, dtype):
    """Largest |error| of an output of this type.

    The output's own rounding, u |out| (u = 2^-8 bf16, 2^-24 fp32). A score is a sum of D <= 128 products in fp32:
    off by at most 128 steps of 2^-24 of its terms' absolute sum E, taken 8 times coarser for the tensor cores'
    accumulation (2^-14 E for bf16, 2^-17 E for fp32); e^s then moves by that share, in numerator and
    denominator: 2. The exponential itself 2^-21. A probability may be rounded to bf16 (2^-8) before the
    product with V. Sums over the keys: keys steps of 2^-24, 8 times coarser on the tensor cores."""
    bf16 = dtype == torch.bfloat16
    u = 2.0 ** -8 if bf16 else 2.0 ** -24
    score = 2 * E * (2.0 ** -14 if bf16 else 2.0 ** -17)
    share = score + 2.0 ** -21 + (2.0 ** -8 if bf16 else 0.0) + 2 * keys * 2.0 ** (-21 if bf16 else -24)
    return u * (out.abs() + share * A) + share * A


def rope(x, cs):
    """x [..., D] in 64 bits turned by cs [..., D / 2, 2] (broadcast)."""
    a, b = x.double().unflatten(-1, (-1, 2)).unbind(-1)
    c, s = cs.double().unbind(-1)
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
