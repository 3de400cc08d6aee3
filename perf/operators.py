"""The paged-serving operators, as cases that can be timed and compared.

One serving step over a paged KV cache: the block tables are extended for the
step's new tokens and every new token gets its cache slot (``tables``), the
new keys and values go into those slots (``write``), and the new tokens
attend to the cache: chunks of many tokens per request (``chunk``) or one or
a few tokens per request (``decode``), with or without a sliding window whose
first keys (sinks) stay visible.

    visible(p, j) = j <= p and (j > p - window or j < sinks)      (causal)
    O = sum_j exp(s_j - LSE) v_j,  s_j = scale * q . k_j,  LSE = ln sum_j exp(s_j)

``own`` False computes each operator from elementary torch operations in 32
bits; True makes the library's calls.  ``exact`` computes the definition in
64 bits, one request and one head at a time.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the tables of one decode step: 128 requests, one new token each, pages of 16
        {"name": "tables_decode_step", "op": "tables", "B": 128, "new_lo": 1, "new_hi": 1, "ctx_lo": 1,
         "ctx_hi": 16383, "page": 16, "lens": 1},
        # admission of many prompts at once: 512 requests, chunks of 1 to 128 tokens, some requests idle
        {"name": "tables_many_chunks", "op": "tables", "B": 512, "new_lo": 0, "new_hi": 128, "ctx_lo": 0,
         "ctx_hi": 8192, "page": 64, "lens": 2},
        # the new keys and values of that decode step (head dim 64, 8 KV heads, f16)
        {"name": "write_decode_step", "op": "write", "tokens": 128, "Hkv": 8, "D": 64, "dtype": "f16", "page": 16,
         "pool": 4096, "padded": 0},
        # the keys and values of a whole prompt of 16384 tokens, the last tokens padding without a slot
        {"name": "write_prompt", "op": "write", "tokens": 16384, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64,
         "pool": 24576, "padded": 7},
        # the smallest chunk call: one request, 33 tokens after 1000 keys
        {"name": "chunk_one_short", "op": "chunk", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 16,
         "new_lo": 33, "new_hi": 33, "ctx_lo": 1000, "ctx_hi": 1000, "causal": True, "window": 0, "sinks": 0,
         "lens": 3},
        # decode rows and chunks in one batch: 1 to 512 new tokens after 0 to 4096 keys
        {"name": "chunk_mixed_batch", "op": "chunk", "B": 24, "Hq": 16, "Hkv": 8, "D": 64, "dtype": "f16",
         "page": 16, "new_lo": 1, "new_hi": 512, "ctx_lo": 0, "ctx_hi": 4096, "causal": True, "window": 0,
         "sinks": 0, "lens": 4},
        # the last 4096 tokens of a 16384-token prompt, 64 query heads over 8 KV heads
        {"name": "chunk_long_prompt", "op": "chunk", "B": 1, "Hq": 64, "Hkv": 8, "D": 128, "dtype": "bf16",
         "page": 64, "new_lo": 4096, "new_hi": 4096, "ctx_lo": 12288, "ctx_hi": 12288, "causal": True, "window": 0,
         "sinks": 0, "lens": 5},
        # head dim 256: four prompts of up to 1000 tokens after up to 4096 keys
        {"name": "chunk_head_dim_256", "op": "chunk", "B": 4, "Hq": 16, "Hkv": 4, "D": 256, "dtype": "bf16",
         "page": 16, "new_lo": 300, "new_hi": 1000, "ctx_lo": 100, "ctx_hi": 4096, "causal": True, "window": 0,
         "sinks": 0, "lens": 6},
        # two prompts with a window of 1024 keys and 4 sinks
        {"name": "chunk_window", "op": "chunk", "B": 2, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 16,
         "new_lo": 2048, "new_hi": 2048, "ctx_lo": 3000, "ctx_hi": 8192, "causal": True, "window": 1024, "sinks": 4,
         "lens": 7},
        # one request, one token, a window of 512 keys and 4 sinks at 4000 keys
        {"name": "decode_window_one", "op": "decode", "B": 1, "q_len": 1, "Hq": 16, "Hkv": 8, "D": 64,
         "dtype": "f16", "page": 16, "len_lo": 4000, "len_hi": 4000, "window": 512, "sinks": 4, "lens": 8},
        # a decode batch over long contexts: 32 requests, window of 4096 keys, 16 sinks
        {"name": "decode_window_batch", "op": "decode", "B": 32, "q_len": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "dtype": "bf16", "page": 16, "len_lo": 1, "len_hi": 16384, "window": 4096, "sinks": 16, "lens": 9},
        # a speculative step of 4 tokens with the same kind of window
        {"name": "decode_window_draft", "op": "decode", "B": 16, "q_len": 4, "Hq": 32, "Hkv": 8, "D": 128,
         "dtype": "bf16", "page": 64, "len_lo": 1023, "len_hi": 8192, "window": 1000, "sinks": 4, "lens": 10},
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "write", "chunk", "chunk", "decode", "decode"])
    lens = rng.randrange(1 << 20)
    if op == "tables":
        B = _log_int(rng, 1, 2048)
        return {"op": op, "B": B, "new_lo": rng.choice([0, 1]), "new_hi": _log_int(rng, 1, max(1, 65536 // B)),
                "ctx_lo": 0, "ctx_hi": _log_int(rng, 1, 16384), "page": rng.choice([8, 16, 24, 32, 64, 128]), "lens": lens}
    if op == "write":
        tokens = _log_int(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "Hkv": rng.choice([1, 2, 4, 5, 8]), "D": rng.choice([64, 128]),
                "dtype": rng.choice(["bf16", "f16"]), "page": rng.choice([8, 16, 32, 64]),
                "pool": tokens + _log_int(rng, 64, 8192), "padded": rng.choice([0, rng.randrange(0, 9)])}
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    case = {"op": op, "B": 1, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "dtype": rng.choice(["bf16", "f16"])}
    if op == "decode":
        lo = rng.choice([1, 1000])
        case.update(B=_log_int(rng, 1, 64), q_len=rng.choice([1, 1, 2, 4]), page=rng.choice([16, 32, 64]), len_lo=lo,
                    len_hi=lo + _log_int(rng, 64, 15000), window=_log_int(rng, 32, 4096), sinks=rng.choice([0, 4, 20, 128]),
                    lens=lens)
        return case
    B = _log_int(rng, 1, 24)
    new = _log_int(rng, 2, 2048)
    ctx = _log_int(rng, 1, 14000)
    # at most the padded size of the largest listed case's scores, and a quarter of its heads times lengths
    while B > 1 and B * Hkv * G * new * (new + ctx) > 1 << 30:
        B -= 1
    windowed = rng.random() < 0.4
    case.update(B=B, page=rng.choice([8, 16, 24, 32, 64, 128]), new_lo=rng.choice([1, max(1, new // 2), new]), new_hi=new,
                ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx, causal=windowed or rng.random() < 0.9,
                window=_log_int(rng, 32, 4096) if windowed else 0, sinks=rng.choice([0, 4, 20, 128]) if windowed else 0,
                lens=lens)
    return case


def _lengths(case):
    """(context keys, new tokens) of every request, from the case alone."""
    r = np.random.default_rng(case["lens"])
    B = case["B"]
    if case["op"] == "decode":
        total = r.integers(case["len_lo"], case["len_hi"] + 1, B)
        new = np.minimum(case["q_len"], total)
        return total - new, new
    ctx = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, B)
    new = r.integers(case["new_lo"], case["new_hi"] + 1, B)
    return ctx, new


def _visible(case):
    """(query-key pairs, distinct keys) that the requests' masks leave, summed over requests."""
    ctx, new = _lengths(case)
    pairs = keys = 0
    window, sinks = case["window"], case["sinks"]
    for c, n in zip(ctx.tolist(), new.tolist()):
        L = c + n
        if case["op"] == "chunk" and not case["causal"]:
            pairs += n * L
            keys += L if n else 0
            continue
        p = np.arange(c, L)
        if window:
            first = np.maximum(0, p - window + 1)
            pairs += int((p - first + 1 + np.minimum(sinks, first)).sum())
            low = max(0, c - window + 1)
            keys += (L - low + min(sinks, low)) if n else 0
        else:
            pairs += int((p + 1).sum())
            keys += L if n else 0
    return pairs, keys


def work(case):
    if case["op"] == "tables":
        ctx, new = _lengths(case)
        page = case["page"]
        taken = int((-(-(ctx + new) // page) - -(-ctx // page)).sum())
        # lengths, offsets, free pages and each request's last held page in; the pages taken, the slots and the lengths out
        n = case["B"] * 4 * 4 + taken * 8 + int(new.sum()) * 4
        return {"bytes": n, "flops": int(new.sum())}
    if case["op"] == "write":
        row = case["Hkv"] * case["D"] * 2
        return {"bytes": case["tokens"] * (4 + 4 * row), "flops": 0}
    pairs, keys = _visible(case)
    _, new = _lengths(case)
    total = int(new.sum()) if case["op"] == "chunk" else case["B"] * case["q_len"]
    rows = total * case["Hq"]
    return {"bytes": rows * (4 * case["D"] + 4) + keys * case["Hkv"] * case["D"] * 4 + -(-keys // case["page"]) * 4,
            "flops": 4 * case["Hq"] * case["D"] * pairs}


# --------------------------------------------------------------- the inputs

def _pages_of(total, page, gen):
    """A block table whose rows hold the pages of `total` keys: a permutation of the pool dealt to the rows in order."""
    need = -(-total // page)
    pool = max(1, int(need.sum()))
    perm = torch.randperm(pool, generator=gen, device="cuda", dtype=torch.int32)
    width = max(1, int(need.max()))
    at = np.concatenate([[0], np.cumsum(need)[:-1]])
    j = torch.arange(width, device="cuda")
    need_t, at_t = (torch.from_numpy(x).cuda() for x in (need, at))
    table = torch.where(j < need_t[:, None], perm[(at_t[:, None] + j).clamp_max(pool - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    return table.to(torch.int32).contiguous(), pool


def _ints(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "tables":
        ctx, new = _lengths(case)
        page, B = case["page"], case["B"]
        have, need = -(-ctx // page), -(-(ctx + new) // page)
        pages = int(need.sum()) + 16  # a few pages stay free
        perm = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
        width = max(1, int(need.max()))
        at = np.concatenate([[0], np.cumsum(have)[:-1]])
        j = torch.arange(width, device="cuda")
        have_t, at_t = torch.from_numpy(have).cuda(), torch.from_numpy(at).cuda()
        held = int(have.sum())
        table = torch.where(j < have_t[:, None], perm[(at_t[:, None] + j).clamp_max(pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
        cu = np.concatenate([[0], np.cumsum(new)])
        state.update(block_table=table.to(torch.int32).contiguous(), free_pages=perm[held:].contiguous(), seqlens=_ints(ctx),
                     cu=_ints(cu), total=int(cu[-1]), num_pages=pages)
        return state
    dtype = DTYPES[case["dtype"]]
    Hkv, D, page = case["Hkv"], case["D"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    if case["op"] == "write":
        n, num_pages = case["tokens"], -(-case["pool"] // page)
        slots = torch.randperm(num_pages, generator=gen, device="cuda", dtype=torch.int64)[:, None] * page + torch.arange(page, device="cuda")
        slots = slots.reshape(-1)[:n].to(torch.int32).contiguous()
        if case["padded"]:
            slots[max(0, n - case["padded"]):] = -1
        state.update(k_new=normal(n, Hkv, D), v_new=normal(n, Hkv, D), slots=slots, k_cache=normal(num_pages, page, Hkv, D),
                     v_cache=normal(num_pages, page, Hkv, D))
        return state
    ctx, new = _lengths(case)
    total = ctx + new
    table, pool = _pages_of(total, page, gen)
    state.update(block_table=table, k_cache=normal(pool, page, Hkv, D), v_cache=normal(pool, page, Hkv, D),
                 seqlens=_ints(total), max_k=int(total.max()))
    if case["op"] == "decode":
        state["q"] = normal(case["B"], case["q_len"], case["Hq"], D)
    else:
        cu = np.concatenate([[0], np.cumsum(new)])
        state.update(q=normal(int(cu[-1]), case["Hq"], D), cu=_ints(cu), max_q=max(1, int(new.max())))
    if own:  # the plan and the workspace that a serving loop keeps
        from decode_attention_packed_b200 import mxa
        if case["op"] == "decode":
            state["prepared"] = mxa.prepare(state["q"], state["k_cache"], table, max_seqlen_k=state["max_k"],
                                            window=case["window"], sinks=case["sinks"])
        else:
            state["prepared"] = mxa.prepare_prefill(state["q"], state["cu"], state["k_cache"], table,
                                                    max_seqlen_q=state["max_q"], max_seqlen_k=state["max_k"])
    return state


# ------------------------------------------------------------ the operators

def run(state):
    if own:
        return _run_own(state)
    return {"tables": _tables, "write": _write, "chunk": _chunk, "decode": _decode}[state["case"]["op"]](state)


def _run_own(state):
    from decode_attention_packed_b200 import mxa
    case = state["case"]
    if case["op"] == "tables":
        slots, seqlens, used = mxa.extend_tables(state["block_table"], state["seqlens"], state["cu"], state["free_pages"],
                                                 page_size=case["page"], num_pages=state["num_pages"], total_q=state["total"])
        return {"block_table": state["block_table"], "slots": slots, "seqlens": seqlens, "used": used}
    if case["op"] == "write":
        mxa.write_cache(state["k_new"], state["v_new"], state["k_cache"], state["v_cache"], state["slots"])
        return {"k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    if case["op"] == "decode":
        out, lse = mxa.decode(state["q"], state["k_cache"], state["v_cache"], state["block_table"], state["seqlens"],
                              causal=True, window=case["window"], sinks=case["sinks"], prepared=state["prepared"])
    else:
        out, lse = mxa.prefill(state["q"], state["cu"], state["k_cache"], state["v_cache"], state["block_table"],
                               state["seqlens"], max_seqlen_q=state["max_q"], causal=case["causal"], window=case["window"],
                               sinks=case["sinks"], prepared=state["prepared"])
    return {"out": out, "lse": lse}


def _tables(state):
    """Pages for the new tokens from the free list in request order, and every new token's slot."""
    page = state["case"]["page"]
    table, ctx, cu, free = state["block_table"], state["seqlens"], state["cu"], state["free_pages"]
    new = cu[1:] - cu[:-1]
    have, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    end = torch.cumsum(need - have, 0, dtype=torch.int32)
    first = end - (need - have)
    j = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)
    taken = (j >= have[:, None]) & (j < need[:, None])
    at = (first[:, None] + j - have[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(taken, free[at], table))
    t = torch.arange(state["total"], device="cuda", dtype=torch.int32)
    row = torch.searchsorted(cu[1:], t, right=True)
    pos = ctx[row] + t - cu[row]
    slots = table[row, pos // page] * page + pos % page
    return {"block_table": table, "slots": slots, "seqlens": ctx + new, "used": end[-1:]}


def _write(state):
    k_cache, v_cache, slots = state["k_cache"], state["v_cache"], state["slots"]
    flat = (-1,) + tuple(k_cache.shape[2:])
    kept = slots >= 0
    at = slots[kept].long()
    k_cache.view(flat)[at] = state["k_new"][kept]
    v_cache.view(flat)[at] = state["v_new"][kept]
    return {"k_cache": k_cache, "v_cache": v_cache}


def _attend(q, limit, low, sinks, state):
    """O [B, Q, Hq, D] and LSE [B, Hq, Q]: query (b, t) sees keys j < limit that are >= low or < sinks (all [B, Q])."""
    case = state["case"]
    B, Q, Hq, D = q.shape
    Hkv, page = case["Hkv"], case["page"]
    G = Hq // Hkv
    L = state["max_k"]
    j = torch.arange(L, device="cuda")
    token = state["block_table"].long()[:, j // page] * page + j % page  # [B, L]; past a row's length any token, masked below
    k = state["k_cache"].view(-1, Hkv, D)[token].float().permute(0, 2, 3, 1)  # [B, Hkv, D, L]
    v = state["v_cache"].view(-1, Hkv, D)[token].float().permute(0, 2, 1, 3)  # [B, Hkv, L, D]
    qg = q.float().view(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    s = (torch.matmul(qg, k) * D ** -0.5).view(B, Hkv, G, Q, L)
    seen = (j < limit[..., None]) & ((j >= low[..., None]) | (j < sinks))  # [B, Q, L]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * Q, L), v).view(B, Hkv, G, Q, D) / l.clamp_min(1e-30)
    out = o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D).to(q.dtype)
    lse = (m + torch.log(l)).view(B, Hq, Q)
    return out, lse


def _decode(state):
    case = state["case"]
    L, n = state["seqlens"].long(), case["q_len"]
    p = L[:, None] - n + torch.arange(n, device="cuda")
    out, lse = _attend(state["q"], (p + 1).clamp_min(0), p - case["window"] + 1, case["sinks"], state)
    return {"out": out, "lse": lse}


def _chunk(state):
    case = state["case"]
    q, cu, L = state["q"], state["cu"].long(), state["seqlens"].long()
    new = cu[1:] - cu[:-1]
    t = torch.arange(state["max_q"], device="cuda")
    p = L[:, None] - new[:, None] + t
    limit = torch.minimum(p + 1, L[:, None]) if case["causal"] else L[:, None].expand_as(p)
    low = p - case["window"] + 1 if case["window"] else torch.zeros_like(p)
    padded = q[(cu[:-1, None] + t).clamp_max(max(0, q.shape[0] - 1))]  # [B, max_q, Hq, D]; past a row's count any query
    out, lse = _attend(padded, limit, low, case["sinks"], state)
    real = t < new[:, None]
    return {"out": out[real], "lse": lse.transpose(1, 2)[real].t().contiguous()}


# ------------------------------------------------------- the exact results

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers
    if case["op"] == "write":
        slots = state["slots"].tolist()
        result = {}
        for name in ("k", "v"):
            cache = state[name + "_cache"].double().cpu()
            flat, fresh = cache.view(-1, *cache.shape[2:]), state[name + "_new"].double().cpu()
            for t, slot in enumerate(slots):
                if slot >= 0:
                    flat[slot] = fresh[t]
            result[name + "_cache"] = cache
        return result
    ctx, new = _lengths(case)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    q = state["q"].view(-1, Hq, D)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    causal = case.get("causal", True)
    start = 0
    for b in range(case["B"]):
        n = case["q_len"] if case["op"] == "decode" else int(new[b])
        length = int(ctx[b] + new[b])
        pages = state["block_table"][b, :-(-length // page)].long()
        keys, values = (state[c][pages].reshape(-1, Hkv, D)[:length].double() for c in ("k_cache", "v_cache"))
        position = torch.arange(length - n, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None]
        hidden = torch.zeros((n, length), dtype=torch.bool, device="cuda")
        if causal:
            hidden = key > position
        if case["window"]:
            hidden |= (key <= position - case["window"]) & (key >= case["sinks"])
        for h in range(Hq if n and length else 0):
            scores = (q[start:start + n, h].double() @ keys[:, h // (Hq // Hkv)].T) / math.sqrt(D)
            scores[hidden] = -math.inf
            total = torch.logsumexp(scores, 1)
            weights = torch.exp(scores - total[:, None])
            weights[torch.isinf(total)] = 0.0
            out[start:start + n, h] = weights @ values[:, h // (Hq // Hkv)]
            lse[h, start:start + n] = total
        start += n
    if case["op"] == "decode":
        B, n = case["B"], case["q_len"]
        return {"out": out.view(B, n, Hq, D), "lse": lse.view(Hq, B, n).transpose(0, 1).contiguous()}
    return {"out": out, "lse": lse}
