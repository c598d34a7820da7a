"""The calls on drafted trees together, as a serving loop makes them: pages for the rows, append,
attention, verify, commit, and forks in between.

The model is a toy whose keys and values depend on a token and its position only, and whose next
token is a function of the present one.  So what must lie in the cache is known at every step: for
each committed position, its token's key turned by that position, to the bit, whatever trees, holes,
forks and page moves came before."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests.attn_harness import assert_close, wide

pytestmark = pytest.mark.gpu

V, D, HKV, HQ, LAYERS, N = 512, 128, 2, 8, 2, 24


def follow(ids):
    """The target's next token."""
    return (ids * 7 + 3) % V


class Loop:
    def __init__(self, page, window=0, sinks=0, B=5, seed=0, num_pages=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.page, self.window, self.sinks, self.B = page, window, sinks, B
        n = lambda *s: torch.randn(s, generator=self.gen, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.k_of, self.v_of, self.q_of = n(LAYERS, V, HKV, D), n(LAYERS, V, HKV, D), 2.0 * n(LAYERS, V, HQ, D)
        self.max_pages = -(-600 // page)
        self.num_pages = num_pages or B * self.max_pages
        self.cache = torch.full((2, LAYERS, self.num_pages, page, HKV, D), float("nan"), dtype=torch.bfloat16,
                                device="cuda")
        self.freq = binding.rope_freq(D)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.tables = [torch.full((B, self.max_pages), -1, **i32) for _ in range(2)]
        view = binding.CacheView(self.cache[0], self.cache[1])
        self.view = view
        self.pages = binding.PageBuffers(view, B_in=B, B=B, max_pages=self.max_pages, sinks=sinks)
        self.rows = B * N
        self.verify = binding.TreeBuffers(B=B, rows=self.rows, q_max=N, V=V)
        self.lens = torch.zeros(B, **i32)          # cached positions
        self.last = torch.tensor(self.rng.integers(0, V, B), **i32)  # the next root
        self.tokens = [[] for _ in range(B)]       # what the cache must hold
        self.zero = torch.zeros(B, **i32)

    def turned(self, ids, pos):
        """Keys of every layer for tokens at positions, by dspark_rope_append."""
        out = []
        for layer in range(LAYERS):
            h = binding.AttnBuffers(B=1, rows=len(ids), q_max=len(ids), Hq=HKV, Hkv=HKV, D=D, rot_dim=D, prompt=True)
            h.bind(q=self.k_of[layer][torch.tensor(ids, device="cuda")].contiguous(),
                   row_req=torch.zeros(len(ids), dtype=torch.int32, device="cuda"),
                   packed_pos=torch.tensor(pos, dtype=torch.int32, device="cuda"), rope_freq=self.freq)
            binding.dspark_rope_append(h.attn)
            out.append(h.q_rot)
        return torch.stack(out)

    def draft(self):
        """Trees of up to N rows: some branches go on as the target does."""
        last = self.last.tolist()
        off, parent, ids = [0], [], []
        for b in range(self.B):
            n = int(self.rng.integers(1, N + 1))
            p, t = [-1], [last[b]]
            for j in range(1, n):
                p.append(int(self.rng.integers(max(0, j - 4), j)))
                t.append(int(follow(t[p[-1]])) if self.rng.random() < 0.6 else int(self.rng.integers(0, V)))
            parent += p
            ids += t
            off.append(off[-1] + n)
        pad = self.rows - off[-1]
        i32 = dict(dtype=torch.int32, device="cuda")
        return (torch.tensor(off, **i32), torch.tensor(parent + [0] * pad, **i32), torch.tensor(ids + [0] * pad, **i32))

    def step(self, parents=None, check=True):
        """``parents``: the requests that each one continues (a fork), or None."""
        if parents is not None:
            at = torch.tensor(parents, device="cuda")
            self.lens, self.last = self.lens[at].clone(), self.last[at].clone()
            self.tokens = [list(self.tokens[p]) for p in parents]
        # pages for the trees' rows; what the window has left is dropped
        first = torch.clamp(self.lens - self.window + 1, min=0) if self.window else None
        parent_t = None if parents is None else torch.tensor(parents, dtype=torch.int32, device="cuda")
        want = self.lens + N
        self.pages.bind(self.tables[0], self.lens, want, parent=parent_t, first_pos=first)
        self.pages.pages.table_out = self.tables[1].data_ptr()
        binding.dspark_update_pages(self.pages.pages)
        self.tables.reverse()
        table = self.tables[0]
        start = self.lens.clone()
        self.before = start.tolist()
        off, parent, ids = self.draft()
        seen, pos, req = binding.tree_rows(parent, off, start)
        outs = []
        for layer in range(LAYERS):
            h = binding.AttnBuffers(B=self.B, rows=self.rows, q_max=N, Hq=HQ, Hkv=HKV, D=D, page_size=self.page,
                                    num_pages=self.num_pages, max_pages=self.max_pages, rot_dim=D, window=self.window)
            at = ids.long()
            h.bind(q=self.q_of[layer][at].contiguous(), k=self.k_of[layer][at].contiguous(),
                   v=self.v_of[layer][at].contiguous(), k_cache=self.cache[0, layer], v_cache=self.cache[1, layer],
                   row_off=off, row_req=req, packed_pos=pos, seq_lens=start, block_table=table, rope_freq=self.freq)
            binding.dspark_rope_append_tree(h.attn)
            binding.dspark_step_attention_tree(h.attn, seen, sinks=self.sinks)
            outs.append(h)
        logits = torch.zeros((self.rows, V), device="cuda")
        logits[torch.arange(self.rows, device="cuda"), follow(ids).long()] = 1.0
        self.verify.bind(logits, off, parent, ids, seq_lens_commit=self.lens)
        binding.dspark_verify_tree(self.verify.tree)
        if check:
            torch.cuda.synchronize()
            self.check_attention(outs, off, seen, pos, start, table)
        binding.dspark_commit_path(self.view.cache, table, start, self.verify.path)
        torch.cuda.synchronize()
        assert self.pages.totals.tolist()[1] == 0 and torch.equal(self.pages.granted_len, want)
        assert self.verify.device_status() == 0 and all(h.device_status() == 0 for h in outs)
        # what was committed: the root and the accepted drafts; the emitted token is the next root
        a, path, out = self.verify.accept_len.tolist(), self.verify.path.tolist(), self.verify.out_tokens.tolist()
        off_h, ids_h, new_last = off.tolist(), ids.tolist(), []
        for b in range(self.B):
            t = [ids_h[off_h[b] + j] for j in path[b][:a[b] + 1]]
            assert t[1:] == out[b][:a[b]] and all(follow(x) == y for x, y in zip(t, t[1:] + [out[b][a[b]]]))
            self.tokens[b] += t
            new_last.append(out[b][a[b]])
        self.last = torch.tensor(new_last, dtype=torch.int32, device="cuda")
        assert self.lens.tolist() == [len(t) for t in self.tokens]
        self.check_cache()
        return a

    def check_cache(self):
        table = self.tables[0].cpu().numpy()
        for b, t in enumerate(self.tokens):
            keep = [p for p in range(len(t)) if not self.window or p > len(t) - self.window or p < self.sinks]
            page, slot = table[b, np.array(keep) // self.page], np.array(keep) % self.page
            assert (page >= 0).all()
            ids = [t[p] for p in keep]
            assert torch.equal(self.cache[0][:, page, slot], self.turned(ids, keep)), b
            assert torch.equal(self.cache[1][:, page, slot], self.v_of[:, torch.tensor(ids, device="cuda")]), b

    def check_attention(self, outs, off, seen, pos, start, table):
        off, start, table = off.cpu().numpy(), start.cpu().numpy(), table.cpu().numpy()
        words, pos = seen.cpu().numpy().view(np.uint64), pos.cpu().numpy()
        layer = LAYERS - 1
        q, out = wide(outs[layer].q_rot), wide(outs[layer].out)
        kc, vc = wide(self.cache[0, layer]), wide(self.cache[1, layer])
        for b in range(self.B):
            r0, r1 = off[b], off[b + 1]
            m = int(start[b]) + r1 - r0
            k, valid = oa.gather(kc, table[b], m)
            v, _ = oa.gather(vc, table[b], m)
            see = oa.seen_tree(int(start[b]), words[r0:r1], pos[r0:r1], m, self.window, self.sinks, valid)
            o, spread, ds = oa.attend_seen(q[r0:r1], np.nan_to_num(k), np.nan_to_num(v), see, D ** -0.5)
            assert_close(out[r0:r1], o, spread, ds, m, b)


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_steps_and_forks(cuda_lib, page, window, sinks):
    loop = Loop(page, window, sinks, seed=page)
    accepted = 0
    for step in range(24):
        parents = None
        if step in (4, 9):
            parents = [int(x) for x in loop.rng.integers(0, loop.B, loop.B)]
        accepted += sum(loop.step(parents, check=step % 5 == 3))
    assert accepted > 40
    used = len(np.unique(loop.tables[0].cpu().numpy())) - 1
    assert loop.pages.totals.tolist()[0] == loop.num_pages - used
    # every page that a position needs is there, and no other: what the window left was freed
    table = loop.tables[0].cpu().numpy()
    for b in range(loop.B):
        kept = loop.before[b]
        first = max(0, kept - window + 1) if window else 0
        for i in range(loop.max_pages):
            needed = i * page < kept + N and ((i + 1) * page > first or i * page < sinks)
            assert (table[b, i] >= 0) == needed, (b, i)
    # (something was left, where pages are no longer than the lengths reached)
    assert not window or page == 64 or max(loop.before) > window + page + sinks


def test_one_request_goes_on_in_many(cuda_lib):
    """All continue one: pages are shared, and each writes a last page of its own."""
    loop = Loop(16, B=6, seed=3)
    for _ in range(4):
        loop.step(check=False)
    loop.step([2] * 6)
    for _ in range(3):
        loop.step()
