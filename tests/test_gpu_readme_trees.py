"""The README's step on drafted trees, as it is printed there: what it commits lies in the cache.

The toy's keys and values depend on the token alone and are not turned, and its next token is a function of
the present one, so every committed position's entries are known to the bit."""
import os
import re

import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests.attn_harness import dev
from tests.test_gpu_step_attention_tree import random_tree

pytestmark = pytest.mark.gpu

V, D, HQ, HKV, LAYERS, B, N = 64, 64, 2, 1, 2, 5, 12


def readme_step():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    block, = [x for x in re.findall(r"```python\n(.*?)```", text, re.S) if "dspark_commit_path" in x]
    return compile(block, "README.md", "exec")


@pytest.mark.parametrize("page", [1, 4, 16])
def test_the_readme_s_step_on_trees(cuda_lib, page):
    step, rng = readme_step(), np.random.default_rng(page)
    max_pages = -(-200 // page)
    num_pages = B * max_pages
    gen = torch.Generator(device="cuda").manual_seed(page)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    cache = torch.full((2, LAYERS, num_pages, page, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    k_of, v_of = n(LAYERS, V, HKV, D), n(LAYERS, V, HKV, D)
    view = binding.CacheView(cache[0], cache[1])
    rows, follow = B * N, lambda x: (x * 5 + 3) % V  # noqa: E731
    names = dict(
        binding=binding, view=view, pages=binding.PageBuffers(view, B_in=B, B=B, max_pages=max_pages),
        tables=[torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda") for _ in range(2)],
        seq_lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
        tree=binding.TreeBuffers(B=B, rows=rows, q_max=N, V=V),
        attn=binding.AttnBuffers(B=B, rows=rows, q_max=N, Hq=HQ, Hkv=HKV, D=D, page_size=page, num_pages=num_pages,
                                 max_pages=max_pages))
    last, tokens, accepted = rng.integers(0, V, B).tolist(), [[] for _ in range(B)], 0
    for _ in range(10):
        count = rng.integers(1, N + 1, B)
        off = np.concatenate([[0], np.cumsum(count)])
        parent, ids = np.zeros(rows, np.int32), np.zeros(rows, np.int32)
        for b in range(B):
            p, at = random_tree(rng, int(count[b]), 0.6), int(off[b])
            parent[at:at + len(p)], ids[at] = p, last[b]
            for j in range(1, len(p)):
                ids[at + j] = follow(ids[at + p[j]]) if rng.random() < 0.7 else rng.integers(0, V)
        t = torch.as_tensor(ids, device="cuda").long()
        logits = torch.zeros((rows, V), device="cuda")
        logits[torch.arange(rows, device="cuda"), follow(t)] = 1.0
        q = n(rows, HQ, D)
        names.update(
            seq_lens_plus_rows=names["seq_lens"] + dev(count.astype(np.int32)), parent=dev(parent),
            row_off=dev(off.astype(np.int32)), packed_ids=dev(ids), target_logits=logits,
            layers=[dict(q=q, k=k_of[i][t], v=v_of[i][t], k_cache=cache[0, i], v_cache=cache[1, i], rope_freq=None)
                    for i in range(LAYERS)])
        exec(step, names)
        torch.cuda.synchronize()
        tree = names["tree"]
        assert torch.equal(names["pages"].granted_len, names["seq_lens_plus_rows"])
        path, emitted, out = tree.path.tolist(), tree.num_emitted.tolist(), tree.out_tokens.tolist()
        for b in range(B):
            tokens[b] += [int(ids[off[b] + j]) for j in path[b][:emitted[b]]]
            last[b] = out[b][emitted[b] - 1]
            accepted += emitted[b] - 1
        assert names["seq_lens"].tolist() == [len(x) for x in tokens]
        table = names["tables"][0].cpu().numpy()
        for b, x in enumerate(tokens):
            pos = np.arange(len(x))
            at = table[b, pos // page], pos % page
            assert (at[0] >= 0).all()
            assert torch.equal(cache[0][:, at[0], at[1]], k_of[:, x]), b
            assert torch.equal(cache[1][:, at[0], at[1]], v_of[:, x]), b
    assert accepted > 10
