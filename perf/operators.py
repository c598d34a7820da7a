"""Measured cases of the attention operators around the verify step.

Three operators on the packed rows of a batch: the position rotation and
append to a paged cache, the attention of a step's rows over that cache, and
the attention of whole prompts.  ``run`` computes them in elementary torch
operations (``own`` false) or through the library (``own`` true).
"""
import math
import random

import torch

own = False

THETA = 1.0e6


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _case(name, op, B, lo, hi, rows_lo=1, rows_hi=1, q_max=1, Hq=32, Hkv=8, D=128, page=64,
          window=0, heads_first=False, interleaved=False, k_rot=False, mix=0):
    """One case.  lo..hi: cached tokens per request before the pass (append, step) or prompt lengths
    (prompt).  rows_lo..rows_hi of q_max packed rows per request.  heads_first: the cache is
    [page, head, slot, D] and not [page, slot, head, D].  mix: seeds the lengths."""
    return {"name": name, "op": op, "B": B, "lo": lo, "hi": hi, "rows_lo": rows_lo,
            "rows_hi": rows_hi, "q_max": q_max, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "window": window, "heads_first": heads_first, "interleaved": interleaved,
            "k_rot": k_rot, "mix": mix}


def listed():
    return [
        # one request's full block of 1 + 16 rows: the latency step at batch 1
        _case("append_step_B1", "append", 1, 2047, 2047, 17, 17, 17, page=16),
        # 256 requests under the batch cap: 1 to 7 of 17 row slots used, the rest is padding
        _case("append_step_B256", "append", 256, 16, 4095, 1, 7, 17, mix=1),
        # prompts entering the batch: whole pages written, rotated keys kept for the prompt's attention
        _case("append_prompts", "append", 8, 0, 0, 501, 4090, 4096, page=16, k_rot=True,
              heads_first=True, mix=2),
        # a single token of a single request: plain decoding, latency counts
        _case("step_decode_B1", "step", 1, 4095, 4095),
        # 32 requests, the full block of 17 rows verified (the static arm), small pages
        _case("step_static_B32", "step", 32, 16, 4095, 17, 17, 17, page=16, mix=3),
        # 256 requests under the batch cap, cached lengths as the step's workloads draw them
        _case("step_mixed_B256", "step", 256, 16, 4095, 1, 7, 17, mix=4),
        # two long contexts, eight query heads per cached head
        _case("step_long_B2", "step", 2, 130000, 131071, 9, 9, 9, Hq=64, heads_first=True, mix=5),
        # sliding window, five query heads per cached head, token-level pages
        _case("step_window_B64", "step", 64, 16, 8191, 1, 17, 17, Hq=40, page=1, window=1024, mix=6),
        # a short question
        _case("prompt_short", "prompt", 1, 77, 77),
        # packed prompts of very different lengths, five query heads per cached head
        _case("prompt_packed_B24", "prompt", 24, 20, 2000, Hq=40, mix=7),
        # one long prompt
        _case("prompt_long", "prompt", 1, 8192, 8192),
        # small heads with a sliding window
        _case("prompt_window_D64", "prompt", 4, 1000, 4100, Hq=16, Hkv=2, D=64, window=512, mix=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "step", "prompt"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    heads = dict(Hq=Hkv * group, Hkv=Hkv, D=D, page=rng.choice([1, 16, 32, 64, 128]),
                 heads_first=rng.random() < 0.5, mix=rng.randrange(1 << 30))
    window = rng.choice([0, 0, _log(rng, 16, 2048)])
    if op == "append":
        if rng.random() < 0.5:  # a step's rows
            q_max = rng.randint(1, 17)
            c = _case("", op, _log(rng, 1, 256), 0, _log(rng, 16, 8192), 1, rng.randint(1, q_max),
                      q_max, **heads)
        else:                   # prompts
            n = _log(rng, 33, 4090)
            c = _case("", op, rng.randint(1, 8), 0, 0, max(1, n // 8), n, n, k_rot=True, **heads)
        c["interleaved"] = rng.random() < 0.3
    elif op == "step":
        q_max = rng.randint(1, 17)
        hi = _log(rng, 16, 65536)
        B = min(_log(rng, 1, 256), max(1, (1 << 19) // hi))
        c = _case("", op, B, rng.randint(0, hi), hi, 1, rng.randint(1, q_max), q_max,
                  window=window, **heads)
    else:
        hi = _log(rng, 33, 8192)
        B = min(rng.randint(1, 24), max(1, (1 << 26) // (hi * hi)))
        c = _case("", op, B, rng.randint(1, hi), hi, window=window, **heads)
        c["Hq"] = min(c["Hq"], 32 // Hkv * Hkv)
    del c["name"]
    return c


def _lengths(case):
    """(cached tokens, packed rows) of each request: fixed by the case, both ends of the ranges among them."""
    r = random.Random(case["mix"])
    B, lo, hi = case["B"], case["lo"], case["hi"]
    ctx = [r.randint(lo, hi) for _ in range(B)]
    ctx[0] = hi
    if B > 1:
        ctx[1] = lo
    rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(B)]
    rows[-1] = case["rows_hi"]
    if case["op"] == "prompt":
        return [0] * B, ctx
    return ctx, rows


def _visible(case):
    """(tokens of the cache or prompt that some row sees, (row, key) pairs seen), summed over the requests."""
    keys = pairs = 0
    W = case["window"]
    for ctx, n in zip(*_lengths(case)):
        first = max(0, ctx + 1 - W) if W else 0
        keys += ctx + n - first
        full = min(n, max(0, W - ctx)) if W else n  # rows whose window reaches the start
        pairs += full * ctx + full * (full + 1) // 2 + (n - full) * W
    return keys, pairs


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    rows = sum(_lengths(case)[1])
    if case["op"] == "append":
        n = rows * D * 2 * (2 * (Hq + 2 * Hkv) + (Hkv if case["k_rot"] else 0))
        return {"bytes": n, "flops": 3 * rows * D * (Hq + Hkv)}
    keys, pairs = _visible(case)
    return {"bytes": (keys * Hkv * D * 2 + rows * Hq * D * 2) * 2, "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, Hq, Hkv, D, page, op = (case[k] for k in ("B", "Hq", "Hkv", "D", "page", "op"))
    ctx, n = _lengths(case)
    used = sum(n)
    rows = used if op == "prompt" or case["rows_hi"] > 64 else B * case["q_max"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731
    off = [0]
    for x in n:
        off.append(off[-1] + x)
    pad = rows - used
    s = {"case": case, "rows": rows, "row_off": i32(off), "seq_lens": i32(ctx),
         "row_req": i32([b for b in range(B) for _ in range(n[b])] + [-1] * pad),
         "row_k": i32([j for b in range(B) for j in range(n[b])] + [-1] * pad),
         "packed_pos": i32([ctx[b] + j for b in range(B) for j in range(n[b])] + [0] * pad),
         "k_cache": None, "v_cache": None, "block_table": None}
    if op != "append":  # rotated queries, of a length that gives scores of standard deviation 2.5
        s["q_rot"] = 2.5 * normal(rows, Hq, D)
    if op == "prompt":  # keys rotated too; values as the projection left them
        s["k_rot"], s["v"] = normal(rows, Hkv, D), normal(rows, Hkv, D)
    else:
        need = [-(-(ctx[b] + n[b]) // page) for b in range(B)]
        num_pages, max_pages = sum(need) + 3, max(need)
        order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
        table, at = torch.zeros((B, max_pages), dtype=torch.int32, device=dev), 0
        for b in range(B):  # pages in no order, as an allocator that has run for a while hands them out
            table[b, : need[b]] = order[at: at + need[b]]
            at += need[b]
        s["block_table"] = table
        shape = (num_pages, Hkv, page, D) if case["heads_first"] else (num_pages, page, Hkv, D)
        for name in ("k_cache", "v_cache"):
            t = normal(*shape) if op == "step" else torch.zeros(shape, dtype=torch.bfloat16, device=dev)
            s[name] = t.transpose(1, 2) if case["heads_first"] else t  # [page, slot, head, D] either way
        if op == "append":  # one projection's output holds q, k and v side by side
            qkv = normal(rows, (Hq + 2 * Hkv) * D)
            s["q"] = qkv[:, : Hq * D].unflatten(1, (Hq, D))
            s["k"] = qkv[:, Hq * D: (Hq + Hkv) * D].unflatten(1, (Hkv, D))
            s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    if own:
        from confidence_driven_speculative_gb300 import binding
        h = binding.AttnBuffers(
            B=B, rows=rows, q_max=max(case["q_max"], max(n)), Hq=Hq, Hkv=Hkv, D=D, page_size=page,
            num_pages=0 if op == "prompt" else num_pages, max_pages=0 if op == "prompt" else max_pages,
            rot_dim=D, interleaved=case["interleaved"], scale=1.0 / math.sqrt(D),
            window=case["window"], k_rot=case["k_rot"], prompt=op == "prompt")
        h.bind(rope_freq=binding.rope_freq(D, THETA, device=dev) if op == "append" else None,
               **{k: s.get(k) for k in ("q", "k", "v", "q_rot", "k_rot", "k_cache", "v_cache",
                                        "row_off", "row_req", "packed_pos", "seq_lens",
                                        "block_table")})
        s["handle"] = h
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        from confidence_driven_speculative_gb300 import binding
        h = state["handle"]
        if op == "append":
            binding.dspark_rope_append(h.attn)
            return _appended(state, h.q_rot, h.k_rot)
        if op == "step":
            binding.dspark_step_attention(h.attn)
        else:
            binding.dspark_prompt_attention(h.attn)
        return h.out
    return {"append": _plain_append, "step": _plain_step, "prompt": _plain_prompt}[op](state)


def _appended(s, q_rot, k_rot):
    out = {"q_rot": q_rot, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["case"]["k_rot"]:
        out["k_rot"] = k_rot
    return out


def _plain_append(s):
    c = s["case"]
    D, page = c["D"], c["page"]
    # far positions: the angle in 64 bits, its sine and cosine rounded to 32
    f = THETA ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    a = s["packed_pos"].double()[:, None] * f
    cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    valid = s["row_req"] >= 0

    def rotate(x):
        x = x.float()
        if c["interleaved"]:
            x0, x1 = x[..., 0::2], x[..., 1::2]
            y = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], dim=-1).flatten(-2)
        else:
            x0, x1 = x[..., : D // 2], x[..., D // 2:]
            y = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], dim=-1)
        return torch.where(valid[:, None, None], y, 0.0).to(torch.bfloat16)

    q_rot, k_rot = rotate(s["q"]), rotate(s["k"])
    at = valid.nonzero()[:, 0]
    pos = s["packed_pos"][at].long()
    pages = s["block_table"][s["row_req"][at].long(), pos // page].long()
    s["k_cache"][pages, pos % page] = k_rot[at]
    s["v_cache"][pages, pos % page] = s["v"][at]
    return _appended(s, q_rot, k_rot)


def _softmax_times(scores, seen, v):
    """softmax over the last axis of the seen scores, times v; rows that see nothing give 0."""
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _plain_step(s):
    c = s["case"]
    B, Hq, Hkv, D, W, n = c["B"], c["Hq"], c["Hkv"], c["D"], c["window"], c["q_max"]
    table = s["block_table"].long()
    # every request's pages side by side: [B, Hkv, keys, D]
    k = s["k_cache"][table].flatten(1, 2).transpose(1, 2).float()
    v = s["v_cache"][table].flatten(1, 2).transpose(1, 2).float()
    j = torch.arange(n, device="cuda")
    rows = s["row_off"][:-1, None].long() + j
    there = rows < s["row_off"][1:, None]
    q = s["q_rot"][rows.clamp(max=s["rows"] - 1)].float()  # [B, n, Hq, D]
    q = q.unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    pos = (s["seq_lens"][:, None] + j)[:, :, None]
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key <= pos) & there[:, :, None]
    if W:
        seen &= key > pos - W
    seen = seen.repeat_interleave(Hq // Hkv, 1)[:, None]
    o = _softmax_times(torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D)), seen, v)
    o = o.unflatten(2, (n, Hq // Hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, n, Hq, D]
    valid = (s["row_req"] >= 0)[:, None, None]
    o = o[s["row_req"].clamp(min=0).long(), s["row_k"].clamp(min=0).long()]
    return torch.where(valid, o, 0.0).to(torch.bfloat16)


def _plain_prompt(s):
    c = s["case"]
    Hq, Hkv, D, W = c["Hq"], c["Hkv"], c["D"], c["window"]
    n = max(_lengths(c)[1])
    j = torch.arange(n, device="cuda")
    rows = (s["row_off"][:-1, None].long() + j).clamp(max=s["rows"] - 1)
    there = s["row_off"][:-1, None] + j < s["row_off"][1:, None]
    q = s["q_rot"][rows].float().unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4)
    k = s["k_rot"][rows].float().transpose(1, 2)[:, :, None]
    v = s["v"][rows].float().transpose(1, 2)[:, :, None]
    seen = j <= j[:, None]
    if W:
        seen &= j > j[:, None] - W
    seen = (seen & there[:, None, :])[:, None, None]
    o = _softmax_times(torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D)), seen, v)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, n, Hq, D]
    return o[s["row_req"].long(), s["row_k"].long()].to(torch.bfloat16)


# --------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, D, Hq, Hkv, W, page = (case[k] for k in ("op", "D", "Hq", "Hkv", "window", "page"))
    off, ctx = s["row_off"].tolist(), s["seq_lens"].tolist()
    if op == "append":
        q_rot = torch.zeros((s["rows"], Hq, D), dtype=torch.float64, device="cuda")
        k_rot = torch.zeros((s["rows"], Hkv, D), dtype=torch.float64, device="cuda")
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        half = D // 2
        for i in range(half):  # one pair of entries at a time
            first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            turn = s["packed_pos"].double() * math.exp(-2.0 * i / D * math.log(THETA))
            z = torch.polar(torch.ones_like(turn), turn)[:, None]
            for x, y in ((s["q"], q_rot), (s["k"], k_rot)):
                w = torch.complex(x[..., first].double(), x[..., second].double()) * z
                y[..., first], y[..., second] = w.real, w.imag
        q_rot[off[-1]:] = 0
        k_rot[off[-1]:] = 0
        for b in range(case["B"]):
            for r0 in range(off[b], off[b + 1], 4096):
                r1 = min(off[b + 1], r0 + 4096)
                p = torch.arange(ctx[b] + r0 - off[b], ctx[b] + r1 - off[b], device="cuda")
                where = s["block_table"][b].long()[p // page]
                kc[where, p % page] = k_rot[r0:r1]
                vc[where, p % page] = s["v"][r0:r1].double()
        return _appended(dict(s, k_cache=kc, v_cache=vc), q_rot, k_rot)
    out = torch.zeros((s["rows"], Hq, D), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        r0, r1 = off[b], off[b + 1]
        end = ctx[b] + r1 - r0
        if op == "step":
            t = torch.arange(end, device="cuda")
            where = s["block_table"][b].long()[t // page]
            k, v = s["k_cache"][where, t % page], s["v_cache"][where, t % page]
        else:
            k, v = s["k_rot"][r0:r1], s["v"][r0:r1]
        t = torch.arange(end, device="cuda")
        i = torch.arange(ctx[b], end, device="cuda")[:, None]
        hidden = (t > i) | (t <= i - W) if W else t > i
        for h in range(Hkv):
            kh, vh = k[:, h].double(), v[:, h].double()
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                x = s["q_rot"][r0:r1, g].double() @ kh.T / math.sqrt(D)
                x[hidden] = -math.inf
                out[r0:r1, g] = torch.softmax(x, -1) @ vh
    return out
