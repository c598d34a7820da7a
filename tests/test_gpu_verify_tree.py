"""dspark_verify_tree against the oracle's walk: everything it writes is whole numbers."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import tree as ot
from tests.attn_harness import dev, offsets
from tests.test_gpu_step_attention_tree import random_tree

pytestmark = pytest.mark.gpu


class Case:
    """Trees whose walks go on with probability ``go`` at each row; the rest of the ids are others.
    ``levels``: logits take that many values only, so that maxima are shared."""

    def __init__(self, seed, n, V, dtype=torch.bfloat16, go=0.8, q_max=None, extra_rows=2, levels=0, deep=0.3):
        rng = np.random.default_rng(seed)
        self.n, self.V, self.B = n, V, len(n)
        self.off, self.rows = offsets(n), sum(n) + extra_rows
        self.q_max = q_max or max(max(n), 1)
        z = rng.integers(0, levels, (self.rows, V)).astype(np.float32) if levels else \
            rng.standard_normal((self.rows, V), np.float32) * 2
        self.z = torch.tensor(z).to(dtype)
        self.logits = self.z.float().numpy()
        self.parent = np.array([p for m in n for p in (random_tree(rng, m, deep) if m else [])]
                               + [0] * extra_rows, np.int32)
        best = self.logits.argmax(1)
        self.ids = rng.integers(0, V, self.rows).astype(np.int32)
        for b in range(self.B):
            at = 0
            while rng.random() < go:
                kids = [j for j in range(1, n[b]) if self.parent[self.off[b] + j] == at]
                if not kids:
                    break
                at, up = int(rng.choice(kids)), at
                self.ids[self.off[b] + at] = best[self.off[b] + up]
        self.lens = rng.integers(0, 1000, self.B).astype(np.int32)

    def handle(self):
        h = binding.TreeBuffers(B=self.B, rows=self.rows, q_max=self.q_max, V=self.V)
        self.commit = dev(self.lens)
        h.bind(self.z.cuda(), dev(self.off), dev(self.parent), dev(self.ids), seq_lens_commit=self.commit)
        return h

    def want(self):
        out = {k: [] for k in ("accept_len", "num_emitted", "path", "out_tokens")}
        for b in range(self.B):
            r0 = self.off[b]
            r1 = min(self.off[b + 1], r0 + self.q_max)
            path, tokens = ot.walk(self.logits[r0:r1], self.parent[r0:r1], self.ids[r0:r1])
            pad = [-1] * (self.q_max - len(path))
            for k, x in (("accept_len", max(len(path) - 1, 0)), ("num_emitted", len(path)), ("path", path + pad),
                         ("out_tokens", tokens + pad)):
                out[k].append(x)
        return {k: np.array(v, np.int32) for k, v in out.items()}

    def check(self, h=None, stream=None, call=True):
        h = h or self.handle()
        if call:
            for k in ("accept_len", "num_emitted", "path", "out_tokens"):
                getattr(h, k).fill_(-7)
            self.commit.copy_(dev(self.lens))
            torch.cuda.synchronize()
            binding.dspark_verify_tree(h.tree, stream)
        torch.cuda.synchronize()
        assert h.device_status() == 0
        want = self.want()
        for k, w in want.items():
            assert np.array_equal(getattr(h, k).cpu().numpy(), w), (k, getattr(h, k).cpu().numpy(), w)
        assert np.array_equal(self.commit.cpu().numpy(), self.lens + want["num_emitted"])
        return want


@pytest.mark.parametrize("V", [8, 24, 1000, 1024, 8192, 32000, 129280])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [[1], [17], [64], [5, 0, 64, 1, 30], [1 + i % 20 for i in range(40)]],
                         ids=["1", "17", "64", "mixed", "many"])
def test_against_the_oracle(cuda_lib, V, dtype, n):
    if V > 100000 and len(n) > 5:
        n = n[:12]
    Case(len(n) + V, n, V, dtype).check()


@pytest.mark.parametrize("B", [150, 300, 700])
def test_many_requests(cuda_lib, B):
    """More walks than there are CTAs at once, and long ones."""
    want = Case(B, [(7 * i) % 33 for i in range(B)], 2048, go=0.9, deep=0.8).check()
    assert want["accept_len"].max() > 8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("levels", [0, 3])
def test_rows_that_a_cta_reads_in_several_rounds(cuda_lib, levels, dtype):
    """So many requests that each has one CTA."""
    Case(6 + levels, [1 + i % 3 for i in range(600)], 17000 if levels else 33000, dtype, levels=levels).check()


def test_a_chain_of_64_rows_accepted_in_full(cuda_lib):
    for V in (1024, 32000):
        c = Case(1, [64, 64], V, deep=1.0, go=1.0)
        assert c.check()["accept_len"].tolist() == [63, 63]


@pytest.mark.parametrize("levels", [1, 2, 7])
@pytest.mark.parametrize("V", [64, 40000])
def test_shared_maxima_go_to_the_lowest_id(cuda_lib, levels, V):
    Case(2, [9, 30, 1, 64], V, levels=levels).check()


@pytest.mark.parametrize("V", [64, 32000])
def test_masked_ids(cuda_lib, V):
    """-inf marks masked ids; a row of nothing else gives the lowest id."""
    c = Case(3, [20, 5], V)
    keep = np.random.default_rng(0).random(c.logits.shape) < 0.1
    c.logits[~keep] = -np.inf
    c.logits[0] = -np.inf
    c.z = torch.tensor(c.logits).to(torch.bfloat16)
    c.logits = c.z.float().numpy()
    c.check()


def test_maxima_at_the_ends_of_a_row(cuda_lib):
    for V in (1000, 129280):
        c = Case(4, [40], V)
        c.logits[:] = np.minimum(c.logits, 3)
        for r in range(40):
            c.logits[r, [0, V - 1, V // 2, V - 8, 7, V // 16, V // 16 - 1, min(4095, V - 2)][r % 8]] = 50.0
        c.z = torch.tensor(c.logits).to(torch.bfloat16)
        c.logits = c.z.float().numpy()
        best = c.logits.argmax(1)
        c.parent[:40] = np.arange(-1, 39)
        c.ids[1:40] = best[:39]
        assert c.check()["accept_len"].tolist() == [39]


def test_children_with_one_token_and_ids_that_are_none(cuda_lib):
    c = Case(5, [6, 4], 1024)
    best = c.logits.argmax(1)
    c.parent[:6] = [-1, 0, 0, 0, 2, 3]
    c.ids[:6] = [0, 5, best[0], best[0], best[2], best[3]]   # rows 2 and 3 both match: 2 goes on
    c.ids[1] = (best[0] + 1) % 1024
    c.parent[6:10] = [-1, 0, 1, 2]
    c.ids[6:10] = [0, -1, 1024, 1 << 30]
    want = c.check()
    assert want["path"][0].tolist() == [0, 2, 4, -1, -1, -1]
    assert want["accept_len"][1] == 0


def test_parents_that_are_none_are_never_reached(cuda_lib):
    c = Case(6, [8], 1024)
    best = c.logits.argmax(1)
    c.parent[:8] = [3, 1, -1, 0, 7, 3, 1 << 30, -(1 << 31)]
    c.ids[:8] = [0, best[0], best[0], best[0], best[7], best[3], best[5], best[5]]
    assert c.check()["path"][0].tolist() == [0, 3, 5, -1, -1, -1, -1, -1]


def test_rows_past_q_max_are_not_there(cuda_lib):
    c = Case(7, [30, 3], 1024, q_max=8, deep=1.0, go=1.0)
    assert c.check()["accept_len"].tolist() == [7, 2]


def test_no_rows_at_all_and_offsets_that_pass_the_rows(cuda_lib):
    c = Case(8, [0, 0], 1024, extra_rows=0)
    h = binding.TreeBuffers(B=2, rows=0, q_max=4, V=1024)
    off = dev(c.off)
    h.tree.logit_dtype, h.tree.row_off = binding.DSPARK_F32, off.data_ptr()
    binding.dspark_verify_tree(h.tree)
    torch.cuda.synchronize()
    assert h.num_emitted.tolist() == [0, 0] and (h.path == -1).all() and (h.out_tokens == -1).all()
    c = Case(9, [5, 9], 1024, extra_rows=0)
    h = c.handle()
    bad = dev(np.array([0, 5, 1 << 30], np.int32))
    h.tree.row_off = bad.data_ptr()
    c.check(h)


def test_far_rows(cuda_lib):
    """Rows whose logits begin past 2^31 elements."""
    V, rows = 1 << 20, 2200
    z = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")
    parent = np.array([j % 22 - 1 for j in range(rows)], np.int32)
    best = np.random.default_rng(1).integers(0, V, rows)
    z[torch.arange(rows, device="cuda"), dev(best)] = 1.0
    ids = np.roll(best, 1).astype(np.int32)
    h = binding.TreeBuffers(B=100, rows=rows, q_max=22, V=V)
    h.bind(z, dev(np.arange(0, rows + 1, 22, dtype=np.int32)), dev(parent), dev(ids))
    binding.dspark_verify_tree(h.tree)
    torch.cuda.synchronize()
    assert (h.accept_len == 21).all()
    assert np.array_equal(h.out_tokens.cpu().numpy().reshape(-1), best)


def test_streams_and_graphs(cuda_lib):
    """One captured call serves other trees and lengths; two run side by side on workspaces of their own."""
    for n, V in (([17], 129280), ([5, 0, 64, 1, 30], 32000)):
        c = Case(10, n, V)
        h = c.handle()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        c.check(h, side.cuda_stream)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            binding.dspark_verify_tree(h.tree, side.cuda_stream)
        other = Case(11, n[::-1], V)
        assert other.rows == c.rows
        for k, x in (("target_logits", other.z), ("row_off", other.off), ("parent", other.parent), ("packed_ids", other.ids)):
            h._keep[k].copy_(x if isinstance(x, torch.Tensor) else dev(x))
        c.commit.copy_(dev(other.lens))
        other.commit = c.commit
        torch.cuda.synchronize()
        g.replay()
        other.check(h, call=False)
    a, b = Case(12, [40] * 9, 32000), Case(13, [40] * 9, 32000)
    ha, hb = a.handle(), b.handle()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(50):
        for h, s in ((ha, streams[0]), (hb, streams[1])):
            h.tree.seq_lens_commit = None
            binding.dspark_verify_tree(h.tree, s.cuda_stream)
    torch.cuda.synchronize()
    for c, h in ((a, ha), (b, hb)):
        for k, w in c.want().items():
            assert np.array_equal(getattr(h, k).cpu().numpy(), w), k


def test_one_workspace_for_every_shape(cuda_lib):
    cases = [Case(20 + i, n, V) for i, (n, V) in enumerate((([30], 4096), ([3, 5, 9], 32000), ([20] * 60, 1024),
                                                             ([64, 1], 512), ([7] * 5, 129280)))]
    handles = [c.handle() for c in cases]
    largest = max(handles, key=lambda h: h.ws_bytes)
    for _ in range(2):
        for c, h in zip(cases, handles):
            h.tree.workspace, h.tree.workspace_bytes = largest.workspace.data_ptr(), largest.ws_bytes
            c.commit = h._keep["seq_lens_commit"]
            c.check(h)
