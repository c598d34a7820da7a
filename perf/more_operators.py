"""Measured cases of the operators for drafted trees, windows with sinks and the cache's pages.

Six operators: the attention of a tree of drafted rows over a paged cache, a
step's and a prompt's attention with a sliding window and first positions that
stay visible (sinks), the verify of a drafted tree, the move of an accepted
path's cache entries to their places, and the pages of a batch's next step
(kept, forked, grown and freed).  ``run`` computes them in elementary torch
operations (``own`` false) or through the library (``own`` true).
"""
import math
import random

import torch

own = False


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _attn(name, op, B, lo, hi, rows_lo=1, rows_hi=1, q_max=1, Hq=32, Hkv=8, D=128, page=64, window=0,
          sinks=0, heads_first=False, mix=0):
    """An attention case.  lo..hi: cached tokens per request (tree, step) or prompt lengths (prompt).
    rows_lo..rows_hi of q_max rows per request.  mix: seeds the lengths and the trees."""
    return {"name": name, "op": op, "B": B, "lo": lo, "hi": hi, "rows_lo": rows_lo, "rows_hi": rows_hi,
            "q_max": q_max, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "window": window, "sinks": sinks,
            "heads_first": heads_first, "mix": mix}


def _verify(name, B, rows_lo, rows_hi, V, f32=False, go=0.7, mix=0):
    """A verify case: trees of rows_lo..rows_hi rows; a walk goes on at a row with probability ``go``."""
    return {"name": name, "op": "verify", "B": B, "rows_lo": rows_lo, "rows_hi": rows_hi, "V": V, "f32": f32,
            "go": go, "mix": mix}


def _commit(name, B, lo, hi, layers, rows=17, go=0.7, Hkv=8, D=128, page=16, heads_first=False, mix=0):
    """A commit case: lo..hi cached tokens per request, trees of ``rows`` rows."""
    return {"name": name, "op": "commit", "B": B, "lo": lo, "hi": hi, "layers": layers, "rows": rows, "go": go,
            "Hkv": Hkv, "D": D, "page": page, "heads_first": heads_first, "mix": mix}


def _pages(name, B_in, fork, lo, hi, grow, layers, done=0.0, window=0, sinks=0, tight=False, Hkv=8, D=128,
           page=16, heads_first=False, mix=0):
    """A pages case: B_in requests of lo..hi tokens, each continued ``fork`` times and grown by ``grow``
    positions; a share ``done`` of the new requests starts from nothing.  tight: fewer pages than wanted."""
    return {"name": name, "op": "pages", "B_in": B_in, "fork": fork, "lo": lo, "hi": hi, "grow": grow,
            "layers": layers, "done": done, "window": window, "sinks": sinks, "tight": tight, "Hkv": Hkv, "D": D,
            "page": page, "heads_first": heads_first, "mix": mix}


def listed():
    return [
        # one request's tree of 60 rows over its context: the latency step at batch 1
        _attn("tree_B1", "tree", 1, 4095, 4095, 60, 60, 60),
        # 32 requests with trees of 17 to 48 rows, cached lengths as the step's workloads draw them, small pages
        _attn("tree_B32", "tree", 32, 16, 4095, 17, 48, 48, page=16, mix=1),
        # a single token of a single request far into its context: latency counts
        _attn("sinks_step_B1", "step", 1, 30000, 30000, window=1024, sinks=4),
        # 256 requests under the batch cap, 1 to 7 rows each, a window of 1024
        _attn("sinks_step_B256", "step", 256, 16, 8191, 1, 7, 17, page=16, window=1024, sinks=4, mix=2),
        # packed prompts of very different lengths, five query heads per cached head
        _attn("sinks_prompt_packed_B24", "prompt", 24, 20, 2000, Hq=40, window=512, sinks=4, mix=3),
        # one long prompt
        _attn("sinks_prompt_long", "prompt", 1, 8192, 8192, window=1024, sinks=64),
        # one request's tree of 32 rows: the latency step at batch 1
        _verify("verify_tree_B1", 1, 32, 32, 129280, mix=4),
        # 128 requests with trees of 9 to 32 rows
        _verify("verify_tree_B128", 128, 9, 32, 129280, mix=5),
        # one request's accepted path through the caches of 32 layers
        _commit("commit_B1", 1, 100, 100, 32, rows=60, go=0.85, mix=33),
        # 256 requests' paths through the caches of 16 layers
        _commit("commit_B256", 256, 5, 40, 16, mix=7),
        # an ordinary step of 256 requests: pages for 17 more rows, some requests replaced
        _pages("pages_step_B256", 256, 1, 16, 4095, 17, 1, done=0.03, Hkv=1, D=64, mix=8),
        # 8 requests forked 8 ways, 32 layers: the last pages are copied
        _pages("pages_fork_B64", 8, 8, 16, 500, 17, 32, page=64, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "step", "prompt", "verify", "commit", "pages"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    mix = rng.randrange(1 << 30)
    place = dict(Hkv=Hkv, D=D, page=rng.choice([1, 12, 16, 32, 64, 128]), heads_first=rng.random() < 0.5, mix=mix)
    if op in ("tree", "step", "prompt"):
        heads = dict(Hq=Hkv * rng.choice([1, 2, 4, 5, 7, 8]), **place)
        sinks = rng.choice([1, 4, 4, 16, 64, _log(rng, 1, 300)])
        window = _log(rng, 16, 4096)
        if op == "prompt":
            hi = _log(rng, 33, 8192)
            B = min(rng.randint(1, 24), max(1, (1 << 26) // (hi * hi)))
            c = _attn("", op, B, rng.randint(1, hi), hi, window=window, sinks=sinks, **heads)
            c["Hq"] = min(c["Hq"], 32 // Hkv * Hkv)
        else:
            q_max = rng.randint(1, 64 if op == "tree" else 17)
            if op == "tree" and rng.random() < 0.6:
                window = sinks = 0
            hi = _log(rng, 16, 65536)
            B = min(_log(rng, 1, 256), max(1, (1 << 18) // hi), max(1, 1024 // q_max))
            c = _attn("", op, B, rng.randint(0, hi), hi, 1, rng.randint(1, q_max), q_max, window=window,
                      sinks=sinks, **heads)
    elif op == "verify":
        V = rng.choice([1024, 32000, 129280, 151936, 8 * _log(rng, 16, 16000)])
        n = rng.randint(1, 64)
        B = min(_log(rng, 1, 256), max(1, 4096 // n))
        c = _verify("", B, rng.randint(1, n), n, V, f32=rng.random() < 0.3, go=rng.random(), mix=mix)
    elif op == "commit":
        B = _log(rng, 1, 256)
        hi = _log(rng, 2, 64)
        c = _commit("", B, rng.randint(0, hi), hi, max(1, min(32, 2048 // B)), rows=rng.randint(1, 32),
                    go=rng.random(), **dict(place, page=min(place["page"], 32)))
    else:
        fork = rng.choice([1, 1, 2, 5, 8])
        B_in = _log(rng, 1, max(1, 256 // fork))
        hi = _log(rng, 2, 4096)
        layers = max(1, min(32, (1 << 15) // (B_in * hi)))
        window = rng.choice([0, 0, _log(rng, 16, 2048)])
        c = _pages("", B_in, fork, rng.randint(1, hi), hi, rng.randint(0, 65), layers, done=rng.choice([0.0, 0.2]),
                   window=window, sinks=rng.choice([0, 4]) if window else 0, tight=rng.random() < 0.2, **place)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# Lengths, trees and paths: fixed by the case
# --------------------------------------------------------------------------
def _tree(r, n):
    """Parents of a tree of n rows, before their children: level by level, or in the order of a search
    that goes on anywhere."""
    p = [-1]
    by_level = r.random() < 0.5
    for j in range(1, n):
        p.append(min(j - 1, max(p[-1], 0) + r.choice([0, 0, 1])) if by_level else r.randrange(j))
    return p


def _depths(p):
    d = [0]
    for j in range(1, len(p)):
        d.append(d[p[j]] + 1)
    return d


def _lengths(case):
    """(cached tokens, rows) of each request, both ends of the ranges among them."""
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


def _trees(case, rows):
    r = random.Random(case["mix"] + 1)
    return [_tree(r, n) for n in rows]


def _walks(case):
    """(parents, rows of the walk after the root) of each request of a verify case."""
    r = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        p = _tree(r, r.randint(case["rows_lo"], case["rows_hi"]))
        at, walk = 0, []
        while r.random() < case["go"]:
            children = [j for j in range(1, len(p)) if p[j] == at]
            if not children:
                break
            at = r.choice(children)
            walk.append(at)
        out.append((p, walk))
    return out


def _paths(case):
    """(cached tokens, accepted rows with the root) of each request of a commit case.  An accepted row lies
    at its place already or behind all places, as level order mostly has it; a pass made twice then gives
    the same."""
    r = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        a = 0
        while r.random() < case["go"] and 2 * (a + 1) < case["rows"]:
            a += 1
        stay = r.randint(0, a) if r.random() < 0.5 else 0
        out.append((r.randint(case["lo"], case["hi"]),
                    list(range(stay + 1)) + sorted(r.sample(range(a + 1, case["rows"]), a - stay))))
    return out


def _plan(case):
    """(lengths of the old requests, parent, kept and wanted lengths and first position of the new ones)."""
    r = random.Random(case["mix"])
    old = [r.randint(case["lo"], case["hi"]) for _ in range(case["B_in"])]
    parent, keep = [], []
    for b in range(case["B_in"] * case["fork"]):
        if r.random() < case["done"]:
            parent.append(-1)
            keep.append(0)
        else:
            parent.append(b // case["fork"])
            n = old[parent[-1]]  # a draft's rejected tail is dropped
            keep.append(max(1, n - r.randint(0, 17)))
    want = [k + case["grow"] if p >= 0 else r.randint(case["lo"], case["hi"]) for p, k in zip(parent, keep)]
    first = [max(0, k - case["window"] + 1) if case["window"] else 0 for k in keep]
    return old, parent, keep, want, first


def _cached(end, pos, case):
    """Of the positions below ``end``, those that a row at ``pos`` sees."""
    W = case["window"]
    lo = max(0, min(end, pos - W + 1)) if W else 0
    return end - lo + min(case["sinks"], lo)


def work(case):
    op = case["op"]
    if op in ("tree", "step", "prompt"):
        keys = pairs = 0
        ctx, rows = _lengths(case)
        trees = _trees(case, rows) if op == "tree" else None
        for b, (c, n) in enumerate(zip(ctx, rows)):
            if op == "tree":
                d = _depths(trees[b])
                keys += _cached(c, c, case) + n
                pairs += sum(_cached(c, c + x, case) + x + 1 for x in d)
            else:
                keys += _cached(c + n, c, case)
                pairs += sum(_cached(p + 1, p, case) for p in range(c, c + n))
        return {"bytes": (keys * case["Hkv"] * 2 + sum(rows) * case["Hq"] * 2) * case["D"] * 2,
                "flops": 4 * case["D"] * case["Hq"] * pairs}
    if op == "verify":  # the rows that the walk comes to
        rows = sum(len(w) + 1 for _, w in _walks(case))
        return {"bytes": rows * case["V"] * (4 if case["f32"] else 2), "flops": rows * case["V"]}
    entry = case["layers"] * 2 * case["Hkv"] * case["D"] * 2
    if op == "commit":
        moved = sum(j != x for _, path in _paths(case) for j, x in enumerate(path))
        named = sum(len(path) for _, path in _paths(case))
        return {"bytes": moved * entry * 2 + named * 8 + case["B"] * 8, "flops": 0}
    old, parent, keep, want, first = _plan(case)
    page, copied, at = case["page"], 0, {}
    for p, k in zip(parent, keep):  # the last pages that two continue to write
        if p >= 0 and k % page and case["grow"]:
            at.setdefault((p, k // page), []).append(k % page)
    copied = sum(sum(x) - x[0] for x in at.values())
    entries = sum(-(-x // page) for x in want)
    return {"bytes": 2 * copied * entry + 8 * entries + 16 * len(parent), "flops": 0}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(n):
    off = [0]
    for x in n:
        off.append(off[-1] + x)
    return _i32(off)


def _cache(case, num_pages, g, layers=None):
    """k and v: [page, slot, head, D] views in either memory order, with the layers in front where there are."""
    lead = () if layers is None else (layers,)
    inner = (case["Hkv"], case["page"]) if case["heads_first"] else (case["page"], case["Hkv"])
    out = []
    for _ in range(2):
        t = torch.randn((*lead, num_pages, *inner, case["D"]), generator=g, device="cuda", dtype=torch.bfloat16)
        out.append(t.transpose(-2, -3) if case["heads_first"] else t)
    return out


def _table(need, num_pages, max_pages, g):
    """Pages in no order, as an allocator that has run for a while hands them out."""
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    need = torch.tensor(need, device="cuda")
    there = torch.arange(max_pages, device="cuda") < need[:, None]
    table = torch.full(there.shape, -1, dtype=torch.int32, device="cuda")
    table[there] = order[: int(need.sum())]
    return table


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op in ("tree", "step", "prompt"):
        B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
        ctx, n = _lengths(case)
        used = sum(n)
        rows = used if op == "prompt" else B * case["q_max"]
        pad = rows - used
        depth = [_depths(p) for p in _trees(case, n)] if op == "tree" else [range(x) for x in n]
        s |= {"rows": rows, "row_off": _offsets(n), "seq_lens": _i32(ctx),
              "row_req": _i32([b for b in range(B) for _ in range(n[b])] + [-1] * pad),
              "row_k": _i32([j for b in range(B) for j in range(n[b])] + [-1] * pad),
              "packed_pos": _i32([ctx[b] + d for b in range(B) for d in depth[b]] + [0] * pad),
              # rotated queries, of a length that gives scores of standard deviation 2.5
              "q_rot": 2.5 * torch.randn((rows, Hq, D), generator=g, device="cuda", dtype=torch.bfloat16)}
        num_pages = max_pages = 0
        if op == "prompt":
            for name in ("k_rot", "v"):
                s[name] = torch.randn((rows, Hkv, D), generator=g, device="cuda", dtype=torch.bfloat16)
        else:
            need = [-(-(ctx[b] + n[b]) // page) for b in range(B)]
            num_pages, max_pages = sum(need) + 3, max(need)
            s["block_table"] = _table(need, num_pages, max_pages, g)
            s["k_cache"], s["v_cache"] = _cache(case, num_pages, g)
        if op == "tree":  # a row sees itself and its ancestors
            seen = []
            for p in _trees(case, n):
                m = [1]
                for j in range(1, len(p)):
                    m.append(m[p[j]] | 1 << j)
                seen += m
            s["row_seen"] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in seen] + [0] * pad,
                                         dtype=torch.int64, device="cuda")
        if own:
            from confidence_driven_speculative_gb300 import binding
            h = binding.AttnBuffers(B=B, rows=rows, q_max=max(n) if op == "prompt" else case["q_max"], Hq=Hq, Hkv=Hkv,
                                    D=D, page_size=page, num_pages=num_pages, max_pages=max_pages,
                                    scale=1.0 / math.sqrt(D), window=case["window"], prompt=op == "prompt")
            h.bind(**{k: s.get(k) for k in ("q_rot", "k_rot", "v", "k_cache", "v_cache", "row_off", "row_req",
                                            "packed_pos", "seq_lens", "block_table")})
            s["handle"] = h
    elif op == "verify":
        V, plan = case["V"], _walks(case)
        n = [len(p) for p, _ in plan]
        rows = sum(n)
        off = [sum(n[:b]) for b in range(len(n))]
        x = torch.randn((rows, V), generator=g, device="cuda", dtype=torch.float32 if case["f32"] else torch.bfloat16)
        x *= 2.0
        x[torch.arange(rows, device="cuda"), torch.randint(0, V, (rows,), generator=g, device="cuda")] += 10.0
        # a walk's rows hold the target's token at the row before, the others another one
        up = torch.tensor([off[b] + max(q, 0) for b, (p, _) in enumerate(plan) for q in p], device="cuda")
        taken = torch.tensor([j in w for p, w in plan for j in range(len(p))], device="cuda")
        other = torch.randint(1, V, (rows,), generator=g, device="cuda")
        s |= {"target_logits": x, "row_off": _offsets(n), "q_max": max(n),
              "parent": _i32([q for p, _ in plan for q in p]), "up": up}
        s["packed_ids"] = torch.where(taken, _first_max(x)[up], (_first_max(x)[up] + other) % V).to(torch.int32)
        if own:
            from confidence_driven_speculative_gb300 import binding
            h = binding.TreeBuffers(B=case["B"], rows=rows, q_max=s["q_max"], V=V)
            h.bind(target_logits=x, row_off=s["row_off"], parent=s["parent"], packed_ids=s["packed_ids"])
            s["handle"] = h
    elif op == "commit":
        plan, page = _paths(case), case["page"]
        need = [-(-(c + case["rows"]) // page) for c, _ in plan]
        num_pages = sum(need) + 3
        s["block_table"] = _table(need, num_pages, max(need), g)
        s["k_cache"], s["v_cache"] = _cache(case, num_pages, g, case["layers"])
        s["seq_lens"] = _i32([c for c, _ in plan])
        s["path"] = _i32([path + [-1] * (case["rows"] - len(path)) for _, path in plan])
        if own:
            from confidence_driven_speculative_gb300 import binding
            s["handle"] = binding.CacheView(s["k_cache"], s["v_cache"])
    else:
        old, parent, keep, want, first = _plan(case)
        page = case["page"]
        need = [-(-x // page) for x in old]
        more = sum(-(-w // page) - (k // page) + 1 for k, w in zip(keep, want))
        num_pages = sum(need) + 3 + (more // 3 if case["tight"] else more)
        max_pages = max(need + [-(-x // page) for x in want])
        s["table_in"] = _table(need, num_pages, max_pages, g)
        s["k_cache"], s["v_cache"] = _cache(case, num_pages, g, case["layers"])
        s |= {"parent": _i32(parent), "keep_len": _i32(keep), "want_len": _i32(want), "first_pos": _i32(first)}
        if own:
            from confidence_driven_speculative_gb300 import binding
            h = binding.PageBuffers(binding.CacheView(s["k_cache"], s["v_cache"]), B_in=len(old), B=len(parent),
                                    max_pages=max_pages, sinks=case["sinks"])
            h.bind(**{k: s[k] for k in ("table_in", "parent", "keep_len", "want_len", "first_pos")})
            s["handle"] = h
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from confidence_driven_speculative_gb300 import binding
        h = state["handle"]
        if op == "tree":
            binding.dspark_step_attention_tree(h.attn, state["row_seen"], sinks=c["sinks"])
            return h.out
        if op == "step":
            binding.dspark_step_attention_sinks(h.attn, c["sinks"])
            return h.out
        if op == "prompt":
            binding.dspark_prompt_attention_sinks(h.attn, c["sinks"])
            return h.out
        if op == "verify":
            binding.dspark_verify_tree(h.tree)
            return {k: getattr(h, k) for k in ("accept_len", "num_emitted", "path", "out_tokens")}
        if op == "commit":
            binding.dspark_commit_path(h.cache, state["block_table"], state["seq_lens"], state["path"])
            return {k: state[k] for k in ("k_cache", "v_cache")}
        binding.dspark_update_pages(h.pages)
        return {"table": h.table_out, "granted": h.granted_len, "tail_src": h.tail_src, "tail_dst": h.tail_dst,
                "totals": h.totals, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    return {"tree": _plain_step, "step": _plain_step, "prompt": _plain_prompt, "verify": _plain_verify,
            "commit": _plain_commit, "pages": _plain_pages}[op](state)


def _softmax_times(scores, seen, v):
    """softmax over the last axis of the seen scores, times v; rows that see nothing give 0."""
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _plain_step(s):
    c = s["case"]
    Hq, Hkv, D, W, n = c["Hq"], c["Hkv"], c["D"], c["window"], c["q_max"]
    table = s["block_table"].clamp(min=0).long()
    # every request's pages side by side: [B, Hkv, keys, D]
    k = s["k_cache"][table].flatten(1, 2).transpose(1, 2).float()
    v = s["v_cache"][table].flatten(1, 2).transpose(1, 2).float()
    j = torch.arange(n, device="cuda")
    rows = s["row_off"][:-1, None].long() + j
    there = rows < s["row_off"][1:, None]
    rows = rows.clamp(max=s["rows"] - 1)
    q = s["q_rot"][rows].float()  # [B, n, Hq, D]
    q = q.unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    pos = s["packed_pos"][rows].long()[:, :, None]
    key = torch.arange(k.shape[2], device="cuda")
    start = s["seq_lens"].long()[:, None, None]
    seen = key < start if c["op"] == "tree" else key <= pos
    if W:
        seen = seen & ((key > pos - W) | (key < c["sinks"]))
    if c["op"] == "tree":
        bit = (key - start).clamp(0, 63)
        drafted = (key >= start) & (key < start + n)
        seen = seen | (drafted & ((s["row_seen"][rows][:, :, None] >> bit) & 1 == 1))
    seen = (seen & there[:, :, None]).repeat_interleave(Hq // Hkv, 1)[:, None]
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
    seen = (j <= j[:, None]) & ((j > j[:, None] - W) | (j < c["sinks"]))
    seen = (seen & there[:, None, :])[:, None, None]
    o = _softmax_times(torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D)), seen, v)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, n, Hq, D]
    return o[s["row_req"].long(), s["row_k"].long()].to(torch.bfloat16)


def _first_max(x):
    """The lowest index of each row's maximum."""
    index = torch.arange(x.shape[1], device=x.device, dtype=torch.int32)
    return torch.where(x == x.amax(1, keepdim=True), index, x.shape[1]).amin(1).long()


def _plain_verify(s):
    c = s["case"]
    B, n = c["B"], s["q_max"]
    best = _first_max(s["target_logits"])
    # the trees side by side, [B, n]; a row that is none is its own parent and no token's
    j = torch.arange(n, device="cuda")
    rows = s["row_off"][:-1, None].long() + j
    there = rows < s["row_off"][1:, None]
    rows = rows.clamp(max=best.shape[0] - 1)
    up = torch.where(there & (j > 0), s["parent"][rows].long(), j)
    y, ids = best[rows], s["packed_ids"][rows].long()
    match = there & (j > 0) & (ids == y.gather(1, up))
    # of a row's children that match, the lowest
    rival = match[:, None, :] & (up[:, None, :] == up[:, :, None]) & (j < j[:, None])
    match &= ~rival.any(2)
    # a row is accepted where it and all of its ancestors match: the ancestors by doubling
    ok = match | (there & (j == 0))
    up = torch.where(j == 0, 0, up)
    for _ in range(6):
        ok = ok & ok.gather(1, up)
        up = up.gather(1, up)
    a = ok.sum(1) - 1
    order = torch.where(ok, j, n).sort(1).values
    path = torch.where(order < n, order, -1)
    last = path.gather(1, a.clamp(min=0)[:, None])
    moved = torch.cat([path[:, 1:], torch.full((B, 1), -1, device="cuda")], 1)
    out = torch.where(moved >= 0, ids.gather(1, moved.clamp(min=0)), -1)
    out = torch.where(j == a[:, None], y.gather(1, last.clamp(min=0)), out)
    return {"accept_len": a.to(torch.int32), "num_emitted": (a + 1).to(torch.int32),
            "path": path.to(torch.int32), "out_tokens": out.to(torch.int32)}


def _plain_commit(s):
    page = s["case"]["page"]
    path, table = s["path"].long(), s["block_table"].long()
    b, j = (path >= 0).nonzero(as_tuple=True)
    src, dst = s["seq_lens"].long()[b] + path[b, j], s["seq_lens"].long()[b] + j
    k, v = s["k_cache"], s["v_cache"]
    moved = [t[:, table[b, src // page], src % page] for t in (k, v)]
    k[:, table[b, dst // page], dst % page] = moved[0]
    v[:, table[b, dst // page], dst % page] = moved[1]
    return {"k_cache": k, "v_cache": v}


def _plain_pages(s):
    c = s["case"]
    page, num_pages = c["page"], s["k_cache"].shape[1]
    table, parent = s["table_in"].long(), s["parent"].long()
    keep, want, first = (s[k].long()[:, None] for k in ("keep_len", "want_len", "first_pos"))
    want = torch.maximum(want, keep)
    i = torch.arange(table.shape[1], device="cuda")
    b = torch.arange(parent.shape[0], device="cuda")[:, None]
    live = (i * page < want) & (((i + 1) * page > first) | (i * page < c["sinks"]))
    old = torch.where((parent >= 0)[:, None], table[parent.clamp(min=0)], -1)
    kept = live & (i * page < keep) & (old >= 0)
    tail = kept & (i == keep // page) & (keep % page != 0) & (want > keep)
    # the lowest request that writes a page goes on with it, where nobody holds it in full
    claim = torch.full((num_pages,), 1 << 30, device="cuda")
    claim.scatter_reduce_(0, old[kept], torch.where(tail, b + 1, 0)[kept], "amin")
    share = tail & (claim[old.clamp(min=0)] != b + 1)
    fresh = live & (i * page >= keep)
    wanted = share | fresh
    rank = (wanted.flatten().cumsum(0) - 1).view(wanted.shape)
    free = (claim == 1 << 30).nonzero()[:, 0]
    given = wanted & (rank < free.shape[0])
    new = torch.cat([free, free.new_zeros(1)])[rank.clamp(0, free.shape[0])]
    out = torch.where(given, new, torch.where(kept, old, -1))
    # the first position that has no memory of its own
    lost = torch.where(wanted & ~given, torch.maximum(i * page, keep), want).amin(1)
    copied = share & given
    src = torch.where(copied, old, -1).amax(1)
    dst = torch.where(copied, new, -1).amax(1)
    slots = torch.arange(page, device="cuda")
    at, slot = (copied.any(1)[:, None] & (slots < keep % page)).nonzero(as_tuple=True)
    s["k_cache"][:, dst[at], slot] = s["k_cache"][:, src[at], slot]
    s["v_cache"][:, dst[at], slot] = s["v_cache"][:, src[at], slot]
    left = torch.stack([(free.shape[0] - wanted.sum()).clamp(min=0), (wanted.sum() - free.shape[0]).clamp(min=0)])
    i32 = torch.int32
    return {"table": out.to(i32), "granted": lost.to(i32), "tail_src": src.to(i32), "tail_dst": dst.to(i32),
            "totals": left.to(i32), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# --------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_attention, "step": _exact_attention, "prompt": _exact_attention,
            "verify": _exact_verify, "commit": _exact_commit, "pages": _exact_pages}[case["op"]](case, s)


def _exact_attention(case, s):
    op, D, Hq, Hkv, W, page = (case[k] for k in ("op", "D", "Hq", "Hkv", "window", "page"))
    off, ctx, pos = s["row_off"].tolist(), s["seq_lens"].tolist(), s["packed_pos"].long()
    if sum(off[b + 1] - off[b] for b in range(case["B"])) * Hq > 1 << 20:
        return None
    out = torch.zeros((s["rows"], Hq, D), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        r0, r1 = off[b], off[b + 1]
        t = torch.arange(ctx[b] + r1 - r0, device="cuda")
        if op == "prompt":
            k, v = s["k_rot"][r0:r1], s["v"][r0:r1]
        else:
            where = s["block_table"][b].long()[t // page]
            k, v = s["k_cache"][where, t % page], s["v_cache"][where, t % page]
        at = pos[r0:r1, None] if op != "prompt" else torch.arange(r1 - r0, device="cuda")[:, None]
        hidden = t > at
        if W:
            hidden = hidden | ((t <= at - W) & (t >= case["sinks"]))
        if op == "tree":
            hidden = hidden | (t >= ctx[b])
            for j, word in enumerate(s["row_seen"][r0:r1].tolist()):
                for i in range(r1 - r0):
                    if word >> i & 1:
                        hidden[j, ctx[b] + i] = False
        for h in range(Hkv):
            kh, vh = k[:, h].double(), v[:, h].double()
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                x = s["q_rot"][r0:r1, g].double() @ kh.T / math.sqrt(D)
                x[hidden] = -math.inf
                out[r0:r1, g] = torch.softmax(x, -1) @ vh
    return out


def _exact_verify(case, s):
    off, parent, ids = s["row_off"].tolist(), s["parent"].tolist(), s["packed_ids"].tolist()
    out = {k: [] for k in ("accept_len", "num_emitted", "path", "out_tokens")}
    for b in range(case["B"]):
        path, tokens = [0], []
        while True:
            r = off[b] + path[-1]
            row = s["target_logits"][r].double()
            y = int((row == row.max()).nonzero()[0])
            children = [j for j in range(1, off[b + 1] - off[b])
                        if parent[off[b] + j] == path[-1] and ids[off[b] + j] == y]
            tokens.append(y)
            if not children:
                break
            path.append(children[0])
        pad = [-1] * (s["q_max"] - len(path))
        for k, x in (("accept_len", len(path) - 1), ("num_emitted", len(path)), ("path", path + pad),
                     ("out_tokens", tokens + pad)):
            out[k].append(x)
    return {k: _i32(x) for k, x in out.items()}


def _exact_commit(case, s):
    page, table, start = case["page"], s["block_table"].tolist(), s["seq_lens"].tolist()
    out = {}
    for name in ("k_cache", "v_cache"):
        new = s[name].double()
        for b, path in enumerate(s["path"].tolist()):
            for j, x in enumerate(path):
                if x >= 0:
                    p, q = start[b] + x, start[b] + j
                    new[:, table[b][q // page], q % page] = s[name][:, table[b][p // page], p % page].double()
        out[name] = new
    return out


def _exact_pages(case, s):
    page, num_pages, table = case["page"], s["k_cache"].shape[1], s["table_in"].tolist()
    parent, keep, want, first = (s[k].tolist() for k in ("parent", "keep_len", "want_len", "first_pos"))
    width = len(table[0])
    out, full, writers = [], set(), {}
    for b, p in enumerate(parent):
        row = [-1] * width
        for i in range(-(-keep[b] // page) if p >= 0 else 0):
            if table[p][i] >= 0 and ((i + 1) * page > first[b] or i * page < case["sinks"]):
                row[i] = table[p][i]
                if want[b] > keep[b] and i * page < keep[b] < (i + 1) * page:
                    writers.setdefault(row[i], []).append(b)
                else:
                    full.add(row[i])
        out.append(row)
    used = full | set(writers)
    free = [x for x in range(num_pages) if x not in used]
    there, asked = len(free), 0
    granted, src, dst = [], [], []
    caches = {k: s[k].double() for k in ("k_cache", "v_cache")}
    for b in range(len(parent)):
        ok, pair = max(want[b], keep[b]), (-1, -1)
        for i in range(-(-max(want[b], keep[b]) // page)):
            x = out[b][i]
            tail = x >= 0 and b in writers.get(x, []) and i == keep[b] // page
            shared = tail and (x in full or writers[x][0] != b)
            fresh = i * page >= keep[b] and ((i + 1) * page > first[b] or i * page < case["sinks"])
            if not shared and not fresh:
                continue
            asked += 1
            if not free:
                ok = min(ok, max(i * page, keep[b]))
                continue
            out[b][i] = free.pop(0)
            if shared:
                pair = (x, out[b][i])
                n = keep[b] % page
                for k, t in caches.items():
                    t[:, pair[1], :n] = s[k][:, pair[0], :n].double()
        granted.append(ok)
        src.append(pair[0])
        dst.append(pair[1])
    return {"table": _i32(out), "granted": _i32(granted), "tail_src": _i32(src), "tail_dst": _i32(dst),
            "totals": _i32([max(0, there - asked), max(0, asked - there)]), **caches}
