"""dspark_update_pages against the oracle: whole numbers and copied entries, so every bit counts."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import tree as ot
from tests.attn_harness import dev, make_table
from tests.test_gpu_commit_path import bits5, make

pytestmark = pytest.mark.gpu


class Case:
    """``B`` requests that continue random ones of ``lens`` (each in pages of its own, and some shared)."""

    def __init__(self, seed, lens, B, page, spare=20, grow=17, window=0, sinks=0, held=False, starts=0.2, layers=2,
                 Hkv=2, D=64, heads_first=False, width=None, forks=True, data=True):
        rng = np.random.default_rng(seed)
        need = [-(-int(n) // page) for n in lens]
        self.page, self.sinks = page, sinks
        self.num_pages = sum(need) + spare
        self.width = width or max(need) + -(-grow // page) + 2
        self.table = make_table(need, self.num_pages, self.width, rng) if len(lens) else np.zeros((0, self.width), np.int32)
        if forks and len(lens) > 2:  # requests that shared pages before
            n = min(need[0], need[1])
            self.table[1, :n] = self.table[0, :n]
        self.parent = np.array([-1 if rng.random() < starts or not len(lens) else int(rng.integers(0, len(lens)))
                                for _ in range(B)], np.int32)
        if not forks:
            self.parent = np.arange(B, dtype=np.int32)
        self.keep = np.array([0 if p < 0 else int(rng.integers(max(0, lens[p] - 20), lens[p] + 1)) for p in self.parent], np.int32)
        self.want = (self.keep + rng.integers(0, grow + 1, B)).astype(np.int32)
        self.first = np.maximum(self.keep - window + 1, 0).astype(np.int32) if window else None
        self.held = (rng.random(self.num_pages) < 0.3).astype(np.int32) if held else None
        self.caches = make(seed, layers, self.num_pages, page, Hkv, D, heads_first) if data else None
        self.B = B

    def handle(self):
        h = binding.PageBuffers(binding.CacheView(*self.caches) if self.caches else None, B_in=len(self.table), B=self.B,
                                max_pages=self.width, sinks=self.sinks, page_size=self.page, num_pages=self.num_pages)
        return h.bind(dev(self.table), dev(self.keep), dev(self.want), parent=None if self.parent is None else dev(self.parent),
                      first_pos=None if self.first is None else dev(self.first),
                      held=None if self.held is None else dev(self.held))

    def want_all(self):
        return ot.update_pages(self.table, self.parent, self.keep, self.want, self.page, self.num_pages, self.first,
                               self.sinks, self.held)

    def check(self, h=None, stream=None, call=True):
        h = h or self.handle()
        want = self.want_all()
        before = [bits5(t) for t in self.caches] if self.caches else []
        if call:
            for k in ("table_out", "granted_len", "tail_src", "tail_dst", "totals"):
                getattr(h, k).fill_(-9)
            torch.cuda.synchronize()
            binding.dspark_update_pages(h.pages, stream)
        torch.cuda.synchronize()
        assert h.device_status() == 0
        for k, w in zip(("table_out", "granted_len", "tail_src", "tail_dst", "totals"), want):
            got = getattr(h, k).cpu().numpy()
            assert np.array_equal(got, w), (k, got, w)
        for t, x in zip(self.caches or (), before):
            for b in range(self.B):
                if want[2][b] >= 0:
                    n = int(min(self.keep[b], self.width * self.page)) % self.page
                    x[:, want[3][b], :n] = x[:, want[2][b], :n]
            assert np.array_equal(bits5(t), x)
        return want


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("B", [1, 6, 40])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 0), (50, 5), (3, 70)])
def test_against_the_oracle(cuda_lib, page, B, window, sinks):
    for seed in range(4):
        Case(seed, [90, 33, 64, 1, 128, 200], B, page, spare=60 * B // page + 20, window=window, sinks=sinks,
             heads_first=seed % 2 == 1).check()


@pytest.mark.parametrize("spare", [0, 1, 5, 30])
@pytest.mark.parametrize("page", [4, 16])
def test_pages_run_out(cuda_lib, spare, page):
    for seed in range(6):
        want = Case(seed, [90, 33, 64, 16, 128, 200], 30, page, spare=spare, grow=40, starts=0.5).check()
    assert spare == 30 or want[4][1] > 0


@pytest.mark.parametrize("page", [1, 16])
def test_held_pages(cuda_lib, page):
    for seed in range(4):
        Case(seed, [90, 33, 64, 1, 128, 200], 20, page, spare=100, held=True).check()


def test_an_ordinary_step(cuda_lib):
    """No fork: every request stays and grows; parent NULL means the same."""
    c = Case(1, [17 * i % 300 + 1 for i in range(100)], 100, 16, spare=300, forks=False)
    c.check()
    c.parent = None
    c.check()


@pytest.mark.parametrize("B,lens,page", [(300, [40] * 30, 16), (2000, [200] * 500, 4), (9000, [3] * 9000, 1),
                                         (20, [20000] * 20, 1), (1, [100000], 1), (3, [9, 9, 9], 65536)])
def test_large_and_small(cuda_lib, B, lens, page):
    Case(2, lens, B, page, spare=20 * B + 40, layers=1, Hkv=1, D=8, grow=9, data=page < 65536).check()


def test_many_pages_few_in_use(cuda_lib):
    Case(3, [50, 60], 5, 16, spare=300000, data=False).check()


def test_a_fork_of_one_into_many(cuda_lib):
    for keep in (32, 33, 47, 48):  # at a page's end, inside, at the next end
        c = Case(4, [48], 64, 16, spare=200, starts=0.0, layers=3, Hkv=3, D=128)
        c.keep[:] = keep
        c.want[:] = keep + 20
        want = c.check()
        assert (want[2] >= 0).sum() == (63 if keep % 16 else 0)


def test_a_reader_keeps_the_writer_off(cuda_lib):
    """The last page of a request that does not grow is not written by one that does."""
    c = Case(5, [40, 40, 40], 2, 16, starts=0.0)
    c.parent[:], c.keep[:], c.want[:] = 2, 40, [60, 40]
    want = c.check()
    assert want[2][0] == c.table[2, 2] and want[3][0] >= 0 and want[0][1, 2] == c.table[2, 2]


def test_odd_arguments(cuda_lib):
    """Lengths and parents out of range, table entries that are none, more than the table takes."""
    c = Case(6, [90, 33, 64, 16], 8, 16, spare=40, window=30)
    c.parent = np.array([-5, 4, 1 << 30, 0, 1, 2, 3, -1], np.int32)
    c.keep = np.array([5, 7, 3, -4, 1 << 30, 60, 16, 2147483647], np.int32)
    c.want = np.array([-1, 20, 2147483647, 12, 0, 70, -9, 3], np.int32)
    c.first = np.array([0, -7, 2147483647, 3, 0, 1 << 30, 2, 5], np.int32)
    c.table[2, 1] = c.num_pages
    c.table[1, 0] = -3
    c.check()


def test_no_requests_before(cuda_lib):
    c = Case(7, [], 5, 16, width=6)
    c.want[:] = [0, 1, 16, 17, 80]
    want = c.check()
    assert (want[0] >= 0).sum() == 0 + 1 + 1 + 2 + 5


def test_without_caches_the_caller_copies(cuda_lib):
    for seed in range(3):
        Case(seed, [90, 33, 64, 1, 128, 200], 12, 16, spare=60, data=False).check()


def test_the_call_again_and_other_shapes_after_it(cuda_lib):
    """The claims are back at zero: the same call gives the same, on a workspace that serves another."""
    a, b = Case(8, [90, 33, 64], 12, 16, spare=90), Case(9, [20, 50, 70, 10], 12, 16, spare=30)
    h = a.handle()
    for _ in range(3):
        a.check(h)
    hb = b.handle()
    hb.pages.workspace, hb.pages.workspace_bytes = h.pages.workspace, h.pages.workspace_bytes
    binding.dspark_workspace_init(h.workspace.data_ptr(), h.ws_bytes)  # another number of pages
    for _ in range(3):
        b.check(hb)


def test_steps_after_steps(cuda_lib):
    """Two tables in turn through 30 steps of growth, forks and ends: pages are never lost or given twice."""
    rng = np.random.default_rng(10)
    B, page, pages, width = 12, 16, 400, 24
    k, v = make(10, 1, pages, page, 1, 8)
    cache = binding.CacheView(k, v)
    tables = [torch.full((B, width), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    h = binding.PageBuffers(cache, B_in=B, B=B, max_pages=width)
    lens = np.zeros(B, np.int32)
    for step in range(30):
        parent = np.array([-1 if rng.random() < 0.1 else int(rng.integers(0, B)) if rng.random() < 0.3 else b
                           for b in range(B)], np.int32)
        keep = np.where(parent >= 0, lens[np.maximum(parent, 0)], 0).astype(np.int32)
        want = np.minimum(keep + rng.integers(0, 18, B), width * page).astype(np.int32)
        host = tables[step % 2].cpu().numpy()
        h.bind(tables[step % 2], dev(keep), dev(want), parent=dev(parent))
        h.pages.table_out = tables[(step + 1) % 2].data_ptr()
        binding.dspark_update_pages(h.pages)
        torch.cuda.synchronize()
        out, granted, _, _, totals = ot.update_pages(host, parent, keep, want, page, pages)
        assert np.array_equal(tables[(step + 1) % 2].cpu().numpy(), out)
        assert np.array_equal(h.granted_len.cpu().numpy(), granted) and h.totals.tolist() == totals.tolist()
        assert totals[0] + len(np.unique(out[out >= 0])) == pages
        lens = want


def test_streams_and_graphs(cuda_lib):
    a, b = Case(11, [90, 33, 64], 12, 16, spare=90, forks=True), Case(12, [90, 33, 64], 12, 16, spare=90)
    assert a.num_pages == b.num_pages and a.width == b.width
    h = a.handle()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.check(h, side.cuda_stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.dspark_update_pages(h.pages, side.cuda_stream)
    for k, x in (("table_in", b.table), ("keep_len", b.keep), ("want_len", b.want), ("parent", b.parent)):
        h._keep[k].copy_(dev(x))
    b.caches = a.caches
    before = [bits5(t) for t in b.caches]
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    want = b.want_all()
    assert np.array_equal(h.table_out.cpu().numpy(), want[0])
    for t, x in zip(b.caches, before):
        for r in range(b.B):
            if want[2][r] >= 0:
                x[:, want[3][r], :b.keep[r] % 16] = x[:, want[2][r], :b.keep[r] % 16]
        assert np.array_equal(bits5(t), x)


def test_one_workspace_for_batches_of_every_size(cuda_lib):
    # every case has the same number of pages; the claims of one call must not count in the next
    cases = [Case(seed, [90, 33, 64], B, 8, spare=100, grow=30) for seed, B in enumerate((3, 70, 1, 200, 12, 70))]
    largest = max((c.handle() for c in cases), key=lambda h: h.ws_bytes)
    for c in cases:
        assert c.num_pages == cases[0].num_pages
        h = c.handle()
        h.workspace, h.ws_bytes = largest.workspace, largest.ws_bytes
        h.pages.workspace, h.pages.workspace_bytes = largest.workspace.data_ptr(), largest.ws_bytes
        c.check(h)
