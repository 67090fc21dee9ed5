"""The paged-serving operators at work: page planning, RoPE with the paged append, and attention over pages and packed prompts.

``own = False`` runs each operator in elementary torch operations, ``own = True`` through
``llama_decoder_block_kv_b200.binding``. A case's request lengths follow from its ``lens`` number alone;
the values of its tensors follow from the seed.
"""
import random

import numpy as np
import torch

own = False

# Model shapes of the repository's workloads: heads, kv heads, head dim, storage type.
SHAPES = {
    "tiny": (4, 2, 64, "fp32"),
    "7b": (32, 32, 128, "bf16"),
    "8b": (32, 8, 128, "bf16"),
    "70b": (64, 8, 128, "bf16"),
}
THETA = 10000.0


def listed():
    return [
        # One decode step of the 8B ragged batch: what a server plans before every token; latency counts.
        {"name": "plan decode 32", "op": "plan", "requests": 32, "single": 32, "new_hi": 1, "kv_lo": 1024, "kv_hi": 8128,
         "page": 16, "lens": 1},
        # An admission wave: many requests with prompts of odd lengths beside running ones.
        {"name": "plan wave 1000", "op": "plan", "requests": 1000, "single": 700, "new_hi": 777, "kv_lo": 0, "kv_hi": 8000,
         "page": 32, "lens": 2},
        # Single tokens of the 8B ragged batch, from the projection's fp32 sums.
        {"name": "append decode 32", "op": "append", "shape": "8b", "in": "fp32", "requests": 32, "single": 32, "new_hi": 1,
         "kv_lo": 1024, "kv_hi": 8128, "page": 16, "lens": 3},
        # A prefill step's worth of prompt chunks at the 70B layer's shape.
        {"name": "append chunks 70b", "op": "append", "shape": "70b", "in": "bf16", "requests": 9, "single": 1,
         "new_hi": 2048, "kv_lo": 0, "kv_hi": 4096, "page": 64, "lens": 4},
        # The 8B ragged decode: one token a request over 1024..8128 cached ones.
        {"name": "paged decode 8b", "op": "paged", "shape": "8b", "requests": 32, "single": 32, "new_hi": 1, "kv_lo": 1024,
         "kv_hi": 8128, "page": 16, "lens": 5},
        # One request of the 7B layer after its 512-token prompt: the smallest call, bound by latency.
        {"name": "paged decode 7b one", "op": "paged", "shape": "7b", "requests": 1, "single": 1, "new_hi": 1, "kv_lo": 512,
         "kv_hi": 640, "page": 64, "lens": 6},
        # Chunked prefill: odd chunks of up to 512 tokens on top of long histories, 8 query heads a kv head.
        {"name": "paged chunks 70b", "op": "paged", "shape": "70b", "requests": 4, "single": 0, "new_hi": 512, "kv_lo": 4096,
         "kv_hi": 8192, "page": 128, "lens": 7},
        # A mixed step: running requests with one token each and a long prompt chunk.
        {"name": "paged mixed 8b", "op": "paged", "shape": "8b", "requests": 24, "single": 22, "new_hi": 2000, "kv_lo": 1024,
         "kv_hi": 8128, "page": 32, "lens": 8},
        # The tiny fp32 model served in chunks.
        {"name": "paged tiny fp32", "op": "paged", "shape": "tiny", "requests": 5, "single": 2, "new_hi": 61, "kv_lo": 3,
         "kv_hi": 700, "page": 16, "lens": 9},
        # The 8B prefill workload, 4 x 8192: the largest.
        {"name": "packed 8b 4x8192", "op": "packed", "shape": "8b", "requests": 4, "single": 0, "new_lo": 8192, "new_hi": 8192,
         "lens": 10},
        # Prompts of odd lengths at the 7B layer's shape (every head its own keys), some of one token.
        {"name": "packed 7b ragged", "op": "packed", "shape": "7b", "requests": 16, "single": 2, "new_lo": 17, "new_hi": 2047,
         "lens": 11},
        # Short prompts of the fp32 model.
        {"name": "packed tiny fp32", "op": "packed", "shape": "tiny", "requests": 7, "single": 1, "new_lo": 5, "new_hi": 509,
         "lens": 12},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "append", "paged", "paged", "packed"])
    c = {"op": op, "lens": rng.randrange(1 << 30)}
    if op == "plan":
        n = _log(rng, 1, 1500)
        return c | {"requests": n, "single": rng.randint(0, n), "new_hi": _log(rng, 1, 900), "kv_lo": 0,
                    "kv_hi": _log(rng, 16, 9000), "page": rng.choice([16, 32, 64, 128])}
    c["shape"] = rng.choice(["tiny", "7b", "8b", "70b"])
    if op == "append":
        n = _log(rng, 1, 64)
        return c | {"in": rng.choice(["fp32", "bf16"]) if c["shape"] != "tiny" else "fp32", "requests": n,
                    "single": rng.randint(0, n), "new_hi": _log(rng, 1, max(1, 12000 // n)), "kv_lo": 0,
                    "kv_hi": _log(rng, 64, 4096), "page": rng.choice([16, 32, 64, 128])}
    if op == "paged":
        n = _log(rng, 1, 40)
        chunk = rng.random() < 0.6
        return c | {"requests": n, "single": rng.randint(0, n) if chunk else n,
                    "new_hi": _log(rng, 2, max(2, min(2048, 8192 // n))) if chunk else 1, "kv_lo": rng.choice([0, 500]),
                    "kv_hi": _log(rng, 512, 8192), "page": rng.choice([16, 32, 64, 128])}
    n = _log(rng, 1, 20)
    hi = _log(rng, 8, 6000 // (1 + n // 4))
    return c | {"requests": n, "single": rng.randint(0, n // 2), "new_lo": 1, "new_hi": hi}


def _lengths(case):
    """(cached, new) tokens of each request: `single` requests of one new token, the others of new_lo..new_hi."""
    r = random.Random(case["lens"])
    n = case["requests"]
    lo = case.get("new_lo", 1)
    new = [1 if b < case["single"] else r.randint(min(lo, case["new_hi"]), case["new_hi"]) for b in range(n)]
    r.shuffle(new)
    cached = [0 if case["op"] == "packed" else r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(n)]
    return cached, new


def _dtype(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _sizes(case):
    cached, new = _lengths(case)
    ps = case["page"]
    pages = [-(-(c + n) // ps) for c, n in zip(cached, new)]
    return cached, new, ps, pages, max(pages) + 1, sum(pages) + 8  # tables a little wider, the pool a little larger than needed


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, dtype):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    s = dict(case)
    if case["op"] == "packed":
        H, Hkv, D, dt = SHAPES[case["shape"]]
        _, new = _lengths(case)
        N = sum(new)
        s.update(H=H, Hkv=Hkv, D=D, new=new, N=N, max_new=max(new), dt=_dtype(dt), max_kv=max(new))
        s["q"], s["k"], s["v"] = (normal((N, h, D), s["dt"]) for h in (H, Hkv, Hkv))
        s["cu"] = _ints(np.concatenate([[0], np.cumsum(new)]).tolist())
        s["out"] = torch.zeros((N, H, D), dtype=s["dt"], device="cuda")
        s["split"] = _split(new, new)
        if own:
            _own_attention(s)
        return s
    cached, new, ps, pages, cols, pool = _sizes(case)
    B, N = len(new), sum(new)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    s.update(cached=_ints(cached), new=_ints(new), B=B, N=N, ps=ps, cols=cols, pool=pool, max_new=max(new),
             max_kv=max(c + n for c, n in zip(cached, new)))
    # Pages already held (those of the cached tokens) come off the front of the permutation; the rest are free.
    held = [-(-c // ps) for c in cached] if case["op"] == "plan" else pages
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(cols, device="cuda", dtype=torch.int64)
    h = torch.tensor(held, device="cuda", dtype=torch.int64)
    start = torch.cumsum(h, 0) - h
    have = col[None, :] < h[:, None]
    table[have] = perm[(start[:, None] + col[None, :])[have]]
    s["table"] = table
    if case["op"] == "plan":
        s["max_tokens"] = N + 5  # a captured step is padded past its tokens
        free = torch.zeros(pool, dtype=torch.int32, device="cuda")
        free[: pool - sum(held)] = perm[sum(held):]
        s["free"], s["free_count"] = free, _ints([pool - sum(held)])
        s["out"] = {k: torch.empty(n, dtype=torch.int32, device="cuda") for k, n in
                    (("cu", B + 1), ("kv", B), ("pos", s["max_tokens"]), ("slot", s["max_tokens"]), ("count", 1))}
        if own:
            from llama_decoder_block_kv_b200 import binding

            s["binding"] = binding
            s["args"] = binding.PageArgs(n_heads=1, n_kv_heads=1, head_dim=64, page_size=ps, num_pages=pool, max_pages=cols)
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    H, Hkv, D, dt = SHAPES[case["shape"]]
    s.update(H=H, Hkv=Hkv, D=D, dt=_dtype(dt))
    s["k_pages"], s["v_pages"] = (normal((pool, Hkv, ps, D), s["dt"]) for _ in range(2))
    kv = torch.tensor([c + n for c, n in zip(cached, new)], device="cuda", dtype=torch.int32)
    if case["op"] == "append":
        s["qkv"] = normal((N, (H + 2 * Hkv) * D), _dtype(case["in"]))
        s["n_pos"] = s["max_kv"] + 1
        inv = THETA ** -(torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        ang = torch.arange(s["n_pos"], dtype=torch.float64, device="cuda")[:, None] * inv
        s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        pos = torch.cat([torch.arange(c, c + n, device="cuda") for c, n in zip(cached, new)])
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), s["new"].long())
        s["pos"] = pos.to(torch.int32)
        s["slot"] = (table[seq, pos // ps] * ps + pos % ps).to(torch.int32)
        s["q_out"] = torch.zeros((N, H, D), dtype=s["dt"], device="cuda")
        if own:
            from llama_decoder_block_kv_b200 import binding

            s["binding"] = binding
            s["args"] = binding.PageArgs(n_heads=H, n_kv_heads=Hkv, head_dim=D, page_size=ps, num_pages=pool, max_pages=cols,
                                         dtype=dt)
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    s["q"] = normal((N, H, D), s["dt"])
    s["cu"] = _ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    s["kv"] = kv
    s["out"] = torch.zeros((N, H, D), dtype=s["dt"], device="cuda")
    s["split"] = _split([c + n for c, n in zip(cached, new)], new)
    if own:
        _own_attention(s)
    return s


def _own_attention(s):
    from llama_decoder_block_kv_b200 import binding

    s["binding"] = binding
    dt = "fp32" if s["dt"] == torch.float32 else "bf16"
    if s["op"] == "paged":
        s["args"] = binding.PageArgs(n_heads=s["H"], n_kv_heads=s["Hkv"], head_dim=s["D"], page_size=s["ps"], num_pages=s["pool"],
                                     max_pages=s["cols"], dtype=dt)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["workspace"] = torch.zeros(binding.llama_attn_workspace_bytes(s["H"], s["Hkv"], s["D"], dt), dtype=torch.uint8, device="cuda")


def _split(kv, new):
    """The requests with one new token and the others, each padded to the longest of its own kind: host-known sizes of the plain form."""
    cu = np.concatenate([[0], np.cumsum(new)])
    parts = []
    for pick in ([b for b, n in enumerate(new) if n == 1], [b for b, n in enumerate(new) if n > 1]):
        if pick:
            t = lambda v: torch.tensor([v[b] for b in pick], device="cuda", dtype=torch.int64)  # noqa: E731
            parts.append({"seq": torch.tensor(pick, device="cuda"), "kv": t(kv), "new": t(new), "start": t(cu.tolist()),
                          "mq": max(new[b] for b in pick), "mk": max(kv[b] for b in pick),
                          "rows": torch.cat([torch.arange(cu[b], cu[b + 1], device="cuda") for b in pick]),
                          "valid": torch.cat([i * max(new[b] for b in pick) + torch.arange(new[x], device="cuda")
                                              for i, x in enumerate(pick)])})
    return parts


def _plain_attention(s, part, k, v, out):
    """softmax(q k^T / sqrt(D)) v over [requests, queries, keys] padded to the longest; k, v: [requests, keys, Hkv, D] in fp32."""
    n, mq, mk = len(part["seq"]), part["mq"], part["mk"]
    H, Hkv, D = s["H"], s["Hkv"], s["D"]
    i = torch.arange(mq, device="cuda")
    rows = part["start"][:, None] + torch.minimum(i[None, :], part["new"][:, None] - 1)
    q = s["q"][rows].float().view(n, mq, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, (H // Hkv) * mq, D)
    p = torch.matmul(q, k.permute(0, 2, 3, 1)).view(n, Hkv, H // Hkv, mq, mk)
    p *= D ** -0.5
    limit = (part["kv"] - part["new"])[:, None] + i[None, :]
    hidden = torch.arange(mk, device="cuda")[None, None, :] > torch.minimum(limit, part["kv"][:, None] - 1)[:, :, None]
    p.masked_fill_(hidden[:, None, None], float("-inf"))
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, Hkv, (H // Hkv) * mq, mk), v.permute(0, 2, 1, 3)).view(n, Hkv, H // Hkv, mq, D)
    o /= total
    o = o.permute(0, 3, 1, 2, 4).reshape(n * mq, H, D)
    out[part["rows"]] = o[part["valid"]].to(out.dtype)


def _plain_plan(s):
    ps, N = s["ps"], s["max_tokens"]
    cached, new = s["cached"].long(), s["new"].long()
    held, kv = (cached + ps - 1) // ps, cached + new
    need = (kv + ps - 1) // ps - held
    before = torch.cumsum(need, 0) - need
    col = torch.arange(s["cols"], device="cuda")[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    at = s["free_count"].long() - 1 - (before[:, None] + col - held[:, None])
    table = torch.where(fresh, s["free"][at.clamp(0, s["pool"] - 1)], s["table"])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(new, 0)])
    t = torch.arange(N, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    inside = seq < s["B"]
    seq = seq.clamp(max=s["B"] - 1)
    pos = cached[seq] + t - cu[seq]
    page = table[seq, (pos // ps).clamp(max=s["cols"] - 1)].long()
    slot = torch.where(inside, page * ps + pos % ps, -1)
    return {"table": table, "cu": cu.int(), "kv": kv.int(), "pos": torch.where(inside, pos, 0).int(), "slot": slot.int(),
            "count": (s["free_count"] - need.sum()).int()}


def _plain_append(s):
    H, Hkv, D, ps = s["H"], s["Hkv"], s["D"], s["ps"]
    x = s["qkv"].float().view(s["N"], H + 2 * Hkv, D // 2, 2)
    c, n = s["rope"][s["pos"].long()].unsqueeze(1).unbind(-1)
    a, b = x[:, : H + Hkv].unbind(-1)
    turned = torch.stack([a * c - b * n, b * c + a * n], -1).view(s["N"], H + Hkv, D)
    s["q_out"].copy_(turned[:, :H])
    page, off = s["slot"].long() // ps, s["slot"].long() % ps
    s["k_pages"][page, :, off] = turned[:, H:].to(s["dt"])
    s["v_pages"][page, :, off] = s["qkv"].view(s["N"], H + 2 * Hkv, D)[:, H + Hkv:].to(s["dt"])
    return s["q_out"], s["k_pages"], s["v_pages"]


def run(s):
    op = s["op"]
    if own:
        b = s["binding"]
        if op == "plan":
            o = s["out"]
            b.llama_page_plan(s["args"], s["cached"], s["new"], s["table"], s["free"], s["free_count"], o["count"], o["cu"], o["kv"],
                              o["pos"], o["slot"], s["status"])
            return {"table": s["table"]} | o
        if op == "append":
            b.llama_rope_append(s["args"], s["qkv"], s["pos"], s["slot"], s["rope"], s["q_out"], s["k_pages"], s["v_pages"], s["status"])
            return s["q_out"], s["k_pages"], s["v_pages"]
        if op == "paged":
            b.llama_attn_paged(s["args"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["kv"], s["max_new"], s["out"],
                               s["workspace"], s["status"])
        else:
            b.llama_attn_packed(s["q"], s["k"], s["v"], s["cu"], s["max_new"], s["out"], s["workspace"], s["status"])
        return s["out"]
    if op == "plan":
        return _plain_plan(s)
    if op == "append":
        return _plain_append(s)
    for part in s["split"]:  # single tokens, then chunks
        j = torch.arange(part["mk"], device="cuda")
        if op == "paged":
            page = s["table"].long()[part["seq"]][:, j // s["ps"]].clamp(min=0)
            k, v = (x[page, :, j % s["ps"]].float() for x in (s["k_pages"], s["v_pages"]))
        else:
            at = part["start"][:, None] + torch.minimum(j[None, :], part["kv"][:, None] - 1)
            k, v = (s[x][at].float() for x in ("k", "v"))
        _plain_attention(s, part, k, v, s["out"])
    return s["out"]


def work(case):
    if case["op"] == "plan":
        cached, new, ps, pages, _, _ = _sizes(case)
        fresh = sum(p - -(-c // ps) for p, c in zip(pages, cached))
        # lengths in, lengths and starts out, a page id read and written, a position and a slot a token
        return {"bytes": 16 * len(new) + 8 * fresh + 8 * (sum(new) + 5), "flops": 0}
    H, Hkv, D, dt = SHAPES[case["shape"]]
    size = 4 if dt == "fp32" else 2
    cached, new = _lengths(case)
    N = sum(new)
    if case["op"] == "append":
        values = (H + 2 * Hkv) * D
        return {"bytes": N * (values * ((4 if case["in"] == "fp32" else 2) + size) + 4 * D + 8), "flops": 3 * N * (H + Hkv) * D}
    kv = [c + n for c, n in zip(cached, new)]
    pairs = sum(c * n + n * (n + 1) // 2 for c, n in zip(cached, new))
    table = 4 * sum(-(-k // case["page"]) for k in kv) if case["op"] == "paged" else 0
    return {"bytes": 2 * size * N * H * D + 2 * size * sum(kv) * Hkv * D + table, "flops": 4 * H * D * pairs}


def exact(case, seed):
    """The operators' definitions, request by request, in 64 bits."""
    s = prepare(case, seed)
    cached, new = _lengths(case)
    if case["op"] == "plan":
        ps, free = s["ps"], s["free"].cpu().numpy()
        top, table = int(s["free_count"]), s["table"].cpu().numpy().copy()
        pos, slot = np.zeros(s["max_tokens"], np.int32), np.full(s["max_tokens"], -1, np.int32)
        t = 0
        for b, (c, n) in enumerate(zip(cached, new)):
            for k in range(-(-c // ps), -(-(c + n) // ps)):
                top -= 1
                table[b, k] = free[top]
            p = np.arange(c, c + n)
            pos[t: t + n], slot[t: t + n] = p, table[b, p // ps] * ps + p % ps
            t += n
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32)  # noqa: E731
        return {"table": i32(table), "cu": i32(np.concatenate([[0], np.cumsum(new)])), "kv": i32(np.add(cached, new)),
                "pos": i32(pos), "slot": i32(slot), "count": i32([top])}
    H, Hkv, D = s["H"], s["Hkv"], s["D"]
    if case["op"] == "append":
        z = s["qkv"].double().view(s["N"], H + 2 * Hkv, D)
        w = torch.view_as_complex(z[:, : H + Hkv].reshape(s["N"], H + Hkv, D // 2, 2).contiguous())
        w = torch.view_as_real(w * torch.view_as_complex(s["rope"].double())[s["pos"].long()][:, None]).flatten(2)
        k, v = s["k_pages"].double(), s["v_pages"].double()
        at = s["slot"].long()
        k.transpose(1, 2).view(s["pool"], s["ps"], Hkv, D)[at // s["ps"], at % s["ps"]] = w[:, H:]
        v.transpose(1, 2).view(s["pool"], s["ps"], Hkv, D)[at // s["ps"], at % s["ps"]] = z[:, H + Hkv:]
        return w[:, :H].contiguous(), k, v
    out = torch.empty((s["N"], H, D), dtype=torch.float64, device="cuda")
    t = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        if case["op"] == "paged":
            ids = s["table"][b, : -(-(c + n) // s["ps"])].long()
            k, v = (x[ids].transpose(1, 2).reshape(-1, Hkv, D)[: c + n] for x in (s["k_pages"], s["v_pages"]))
        else:
            k, v = s["k"][t: t + n], s["v"][t: t + n]
        visible = torch.ones((n, c + n), dtype=torch.bool, device="cuda").tril(c)
        for h in range(H):
            g = h // (H // Hkv)
            a = (s["q"][t: t + n, h].double() @ k[:, g].double().T) / D ** 0.5
            a = torch.softmax(torch.where(visible, a, -torch.inf), -1)
            out[t: t + n, h] = a @ v[:, g].double()
        t += n
    return out
