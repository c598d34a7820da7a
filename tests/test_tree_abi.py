"""CPU checks of the calls on trees, windows with sinks and the caches' pages: the structs' layout,
the refusals (all on the host, before the GPU is touched), the binding's own checks and set-up."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import _build, binding
from oracle import tree as ot
from tests.test_attn_abi import FAKE, ROOT, fake, valid

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE = (binding.DSPARK_OK, binding.DSPARK_EINVAL, binding.DSPARK_EDTYPE,
                                          binding.DSPARK_EALIGN, binding.DSPARK_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def filled(cls, **kw):
    a = cls()
    for name, kind in cls._fields_:
        if kind is ctypes.c_void_p:
            setattr(a, name, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def tree(**kw):
    t = filled(binding.DsparkTree, B=4, rows=36, q_max=9, V=1024, logit_dtype=binding.DSPARK_BF16,
               workspace_bytes=binding.dspark_tree_workspace_size(4, 36, 1024))
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def cache(**kw):
    c = filled(binding.DsparkCache, layers=3, Hkv=2, D=128, dtype=binding.DSPARK_BF16, page_size=16, num_pages=64,
               layer_stride=64 * 16 * 256, page_stride=16 * 256, slot_stride=256, head_stride=128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def pages(**kw):
    p = filled(binding.DsparkPages, cache=cache(), B_in=4, B=4, max_pages=8, sinks=0, table_out=2 * FAKE,
               workspace_bytes=binding.dspark_pages_workspace_size(4, 64))
    for k, v in kw.items():
        setattr(p if hasattr(p, k) else p.cache, k, v)
    return p


@pytest.mark.parametrize("cls,name", [(binding.DsparkTree, "dspark_tree"), (binding.DsparkCache, "dspark_cache"),
                                      (binding.DsparkPages, "dspark_pages")])
def test_struct_layout_matches_c(lib, cls, name):
    fields = [f for f, _ in cls._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "dspark.h"', "int main(void){",
           f'printf("%zu\\n", sizeof({name}));']
    src += [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields] + ["return 0;}"]
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "layout.c"), os.path.join(td, "layout")
        open(c, "w").write("\n".join(src))
        subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                        c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert int(out[0]) == ctypes.sizeof(cls)
    assert [int(x) for x in out[1:]] == [getattr(cls, f).offset for f in fields]


ATTN = {"dspark_rope_append_tree": lambda lib, a: lib.dspark_rope_append_tree(ctypes.byref(a), None),
        "dspark_step_attention_sinks": lambda lib, a: lib.dspark_step_attention_sinks(ctypes.byref(a), 4, None),
        "dspark_prompt_attention_sinks": lambda lib, a: lib.dspark_prompt_attention_sinks(ctypes.byref(a), 4, None),
        "dspark_step_attention_tree": lambda lib, a: lib.dspark_step_attention_tree(ctypes.byref(a), FAKE, 4, None)}


@pytest.mark.parametrize("call", ATTN)
def test_attention_shapes_refused(lib, call):
    for kw in (dict(B=-1), dict(B=65537), dict(rows=-1), dict(q_max=0), dict(Hq=8, Hkv=3), dict(D=96),
               dict(window=-1)):
        assert ATTN[call](lib, valid(**kw)) == EINVAL, kw
        assert call in binding.last_error()
    assert ATTN[call](lib, valid(dtype=7)) == EDTYPE
    for kw in (dict(B=0), dict(rows=0)):
        assert ATTN[call](lib, valid(**kw)) == OK


@pytest.mark.parametrize("call", list(ATTN)[1:])
def test_attention_refusals(lib, call):
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(q_rot=None), dict(row_off=None), dict(out=None)):
        assert ATTN[call](lib, valid(window=64, **kw)) == EINVAL, kw
    assert ATTN[call](lib, valid(out=FAKE + 8)) == EALIGN
    for kw in (dict(workspace=None), dict(workspace=FAKE + 16), dict(workspace_bytes=8)):
        assert ATTN[call](lib, valid(**kw)) == EWORKSPACE, kw


def test_sinks_refused(lib):
    a = valid(window=64)
    assert lib.dspark_step_attention_sinks(ctypes.byref(a), -1, None) == EINVAL
    assert "sinks=-1" in binding.last_error()
    assert lib.dspark_prompt_attention_sinks(ctypes.byref(a), -5, None) == EINVAL
    assert lib.dspark_step_attention_tree(ctypes.byref(a), FAKE, -1, None) == EINVAL
    for f in (lib.dspark_step_attention_sinks, lib.dspark_prompt_attention_sinks):
        assert f(None, 4, None) == EINVAL


def test_tree_attention_refusals(lib):
    f = lib.dspark_step_attention_tree
    assert f(None, FAKE, 0, None) == EINVAL
    assert f(ctypes.byref(valid()), None, 0, None) == EINVAL
    assert "row_seen" in binding.last_error()
    assert f(ctypes.byref(valid()), FAKE + 4, 0, None) == EALIGN
    size = binding.dspark_attn_workspace_size(8, 2, 128, 65)
    assert f(ctypes.byref(valid(q_max=65, workspace_bytes=size)), FAKE, 0, None) == EINVAL
    assert "64" in binding.last_error()
    assert f(ctypes.byref(valid(window=9, packed_pos=None)), FAKE, 0, None) == EINVAL
    for kw in (dict(k_cache=None), dict(block_table=None), dict(page_size=0), dict(max_pages=1 << 30)):
        assert f(ctypes.byref(valid(**kw)), FAKE, 0, None) == EINVAL, kw


def test_tree_append_refusals(lib):
    f = ATTN["dspark_rope_append_tree"]
    for kw in (dict(row_off=None), dict(row_req=None), dict(packed_pos=None), dict(v=None), dict(rot_dim=24)):
        assert f(lib, valid(**kw)) == EINVAL, kw


def test_verify_tree_refusals(lib):
    f = lambda **kw: lib.dspark_verify_tree(ctypes.byref(tree(**kw)), None)  # noqa: E731
    assert lib.dspark_verify_tree(None, None) == EINVAL
    for kw in (dict(B=-1), dict(B=65537), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(q_max=0), dict(q_max=65),
               dict(V=0), dict(V=(1 << 24) + 8), dict(target_logits=None), dict(row_off=None), dict(parent=None),
               dict(packed_ids=None), dict(accept_len=None), dict(num_emitted=None), dict(path=None),
               dict(out_tokens=None)):
        assert f(**kw) == EINVAL, kw
        assert "dspark_verify_tree" in binding.last_error()
    assert f(logit_dtype=5) == EDTYPE
    assert f(target_logits=FAKE + 8) == EALIGN
    assert f(V=1020) == EALIGN
    for kw in (dict(workspace=None), dict(workspace=FAKE + 16), dict(workspace_bytes=8)):
        assert f(**kw) == EWORKSPACE, kw
    assert f(B=0) == OK


def test_commit_path_refusals(lib):
    def f(c, B=4, q_max=9, max_pages=8, table=FAKE, lens=FAKE, path=FAKE):
        return lib.dspark_commit_path(ctypes.byref(c), B, q_max, max_pages, table, lens, path, None)
    assert lib.dspark_commit_path(None, 4, 9, 8, FAKE, FAKE, FAKE, None) == EINVAL
    for kw in (dict(layers=0), dict(layers=1025), dict(Hkv=0), dict(Hkv=257), dict(D=0), dict(D=12), dict(D=520),
               dict(page_size=0), dict(page_size=65537), dict(num_pages=0), dict(k_cache=None), dict(v_cache=None),
               dict(layer_stride=0), dict(slot_stride=-8)):
        assert f(cache(**kw)) == EINVAL, kw
        assert "dspark_commit_path" in binding.last_error()
    for kw in (dict(k_cache=FAKE + 8), dict(v_cache=FAKE + 2), dict(layer_stride=4100), dict(head_stride=132)):
        assert f(cache(**kw)) == EALIGN, kw
    assert f(cache(dtype=binding.DSPARK_F32)) == EDTYPE
    for kw in (dict(B=-1), dict(B=65537), dict(q_max=0), dict(q_max=66), dict(max_pages=0), dict(max_pages=1 << 30),
               dict(table=None), dict(path=None)):
        assert f(cache(), **kw) == EINVAL, kw
    assert f(cache(), B=0) == OK


def test_update_pages_refusals(lib):
    f = lambda **kw: lib.dspark_update_pages(ctypes.byref(pages(**kw)), None)  # noqa: E731
    assert lib.dspark_update_pages(None, None) == EINVAL
    for kw in (dict(B=-1), dict(B=65537), dict(B_in=-1), dict(sinks=-1), dict(max_pages=0), dict(page_size=0),
               dict(num_pages=0), dict(max_pages=1 << 30), dict(k_cache=None), dict(v_cache=None), dict(layers=0),
               dict(table_in=None), dict(keep_len=None), dict(want_len=None), dict(table_out=None),
               dict(granted_len=None), dict(tail_src=None), dict(tail_dst=None), dict(totals=None),
               dict(table_out=FAKE)):
        assert f(**kw) == EINVAL, kw
        assert "dspark_update_pages" in binding.last_error()
    assert f(k_cache=FAKE + 8) == EALIGN
    for kw in (dict(workspace=None), dict(workspace=FAKE + 16), dict(workspace_bytes=8)):
        assert f(**kw) == EWORKSPACE, kw
    assert f(B=0) == OK


def test_workspace_sizes(lib):
    assert binding.dspark_tree_workspace_size(4, 36, 1024) >= 256
    assert binding.dspark_pages_workspace_size(4, 64) >= 256
    for bad in ((-1, 1, 8), (65537, 1, 8), (1, -1, 8), (1, 1, 0), (1, (1 << 24) + 1, 8)):
        assert binding.dspark_tree_workspace_size(*bad) == 0, bad
    for bad in ((-1, 1), (65537, 1), (1, 0)):
        assert binding.dspark_pages_workspace_size(*bad) == 0, bad


def test_tree_rows_against_a_walk_up():
    rng = np.random.default_rng(0)
    for _ in range(20):
        n = [int(x) for x in rng.integers(0, 65, 5)]
        off = np.concatenate([[0], np.cumsum(n)])
        rows = int(off[-1]) + 3
        parent = np.full(rows, 7, np.int32)
        for b in range(5):
            for j in range(n[b]):  # chains, bushes, and parents that are none
                parent[off[b] + j] = rng.choice([j - 1, rng.integers(0, max(j, 1)), -1, j, 99], p=[.5, .3, .1, .05, .05])
        lens = rng.integers(0, 100, 5)
        seen, pos, req = binding.tree_rows(torch.tensor(parent), torch.tensor(off, dtype=torch.int32),
                                           torch.tensor(lens, dtype=torch.int32))
        for b in range(5):
            for j in range(n[b]):
                word, depth, at = 1 << j, 0, j
                while at > 0 and 0 <= parent[off[b] + at] < at:
                    at = int(parent[off[b] + at])
                    word |= 1 << at
                    depth += 1
                r = off[b] + j
                assert int(seen[r]) % (1 << 64) == word
                assert (int(pos[r]), int(req[r])) == (lens[b] + depth, b)
        assert (req[off[-1]:] == -1).all() and (seen[off[-1]:] == 0).all()


def test_binding_checks_what_it_is_given(lib):
    a = valid()
    words = fake(36, dtype=torch.int64)
    for bad, what in ((words.int(), "int64"), (words[:35], "36 elements"), (torch.zeros(36, dtype=torch.int64), "CUDA"),
                      (None, "torch tensor")):
        with pytest.raises(ValueError, match=what):
            binding.dspark_step_attention_tree(a, bad)
    c = cache()
    with pytest.raises(ValueError, match="path must be a matrix"):
        binding.dspark_commit_path(c, fake(4, 8, dtype=torch.int32), None, fake(36, dtype=torch.int32))
    with pytest.raises(ValueError, match="block_table must be"):
        binding.dspark_commit_path(c, fake(3, 8, dtype=torch.int32), None, fake(4, 9, dtype=torch.int32))
    k = fake(3, 64, 16, 2, 128)
    v = binding.CacheView(k, k).cache
    assert (v.layers, v.num_pages, v.page_size, v.Hkv, v.D) == (3, 64, 16, 2, 128)
    assert (v.layer_stride, v.page_stride, v.slot_stride, v.head_stride) == (64 * 4096, 4096, 256, 128)
    one = binding.CacheView(k[0].transpose(1, 2), k[0].transpose(1, 2)).cache
    assert (one.layers, one.page_size, one.Hkv, one.slot_stride, one.head_stride) == (1, 2, 16, 128, 256)
    with pytest.raises(ValueError, match="same strides"):
        binding.CacheView(k, fake(3, 64, 2, 16, 128).transpose(2, 3))
    with pytest.raises(ValueError, match="entries"):
        binding.CacheView(k.transpose(3, 4), k.transpose(3, 4))
    with pytest.raises(ValueError, match="layers, num_pages"):
        binding.CacheView(k[0, 0], k[0, 0])


def test_oracle_of_the_pages():
    """By hand: pages of 4; request 0 of 6 positions in pages 7, 3 is continued three times."""
    table = np.array([[7, 3, -1, -1], [1, 5, 2, -1]], np.int32)
    out, granted, src, dst, totals = ot.update_pages(table, [0, 0, 0, 1, -1], [6, 6, 4, 9, 0], [8, 9, 5, 9, 3], 4, 10)
    #   0 goes on in page 3, 1 copies it to 0 and gets 4, 2 keeps page 7 and gets 6; 3 reads only; 4 starts with 8
    assert out.tolist() == [[7, 3, -1, -1], [7, 0, 4, -1], [7, 6, -1, -1], [1, 5, 2, -1], [8, -1, -1, -1]]
    assert granted.tolist() == [8, 9, 5, 9, 3]
    assert (src.tolist(), dst.tolist()) == ([-1, 3, -1, -1, -1], [-1, 0, -1, -1, -1])
    assert totals.tolist() == [1, 0]


def test_oracle_of_the_walk():
    z = np.array([[0, 3, 3], [9, 0, 0], [0, 0, 1]])
    assert ot.walk(z, [-1, 0, 1], [0, 1, 0]) == ([0, 1, 2], [1, 0, 2])
    assert ot.walk(z, [-1, 0, 0], [0, 2, 1]) == ([0, 2], [1, 2])
    assert ot.walk(z[:0], [], []) == ([], [])
