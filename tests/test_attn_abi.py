"""CPU checks of the attention calls: the struct's layout and the refusals,
which all happen on the host before the GPU is touched."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from confidence_driven_speculative_gb300 import _build, binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # a 256-aligned non-null address; validation never dereferences it
CALLS = ["dspark_rope_append", "dspark_step_attention", "dspark_prompt_attention"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def valid(**kw):
    a = binding.DsparkAttn()
    for name, kind in binding.DsparkAttn._fields_:
        if kind is ctypes.c_void_p:
            setattr(a, name, FAKE)
    a.B, a.rows, a.q_max, a.Hq, a.Hkv, a.D = 4, 36, 9, 8, 2, 128
    a.dtype, a.page_size, a.num_pages, a.max_pages = binding.DSPARK_BF16, 16, 64, 8
    a.rot_dim, a.window, a.scale = 128, 0, 0.1
    a.q_stride, a.k_stride, a.v_stride = 12 * 128, 12 * 128, 12 * 128
    a.page_stride, a.slot_stride, a.head_stride = 16 * 2 * 128, 2 * 128, 128
    a.workspace_bytes = binding.dspark_attn_workspace_size(8, 2, 128, 9)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def status(lib, call, a):
    return getattr(lib, call)(ctypes.byref(a), None)


def test_struct_layout_matches_c(lib):
    fields = [f for f, _ in binding.DsparkAttn._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "dspark.h"', "int main(void){",
           'printf("%zu\\n", sizeof(dspark_attn));']
    src += [f'printf("%zu\\n", offsetof(dspark_attn, {f}));' for f in fields] + ["return 0;}"]
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "layout.c"), os.path.join(td, "layout")
        open(c, "w").write("\n".join(src))
        subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                        c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert int(out[0]) == ctypes.sizeof(binding.DsparkAttn)
    assert [int(x) for x in out[1:]] == [getattr(binding.DsparkAttn, f).offset for f in fields]


def test_workspace_size(lib):
    assert binding.dspark_attn_workspace_size(8, 2, 128, 9) > 0
    assert binding.dspark_attn_workspace_size(8, 2, 64, 100000) > 0
    for bad in ((0, 1, 128, 1), (8, 3, 128, 1), (2, 4, 128, 1), (257, 1, 128, 1), (8, 2, 96, 1),
                (8, 2, 128, 0)):
        assert binding.dspark_attn_workspace_size(*bad) == 0, bad


@pytest.mark.parametrize("call", CALLS)
def test_shapes_refused_by_every_call(lib, call):
    assert getattr(lib, call)(None, None) == binding.DSPARK_EINVAL
    assert "NULL" in binding.last_error()
    for kw in (dict(B=-1), dict(B=65537), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(q_max=0),
               dict(Hq=0), dict(Hkv=0), dict(Hq=8, Hkv=3), dict(Hq=2, Hkv=4), dict(Hq=512),
               dict(D=0), dict(D=96), dict(D=256), dict(window=-1)):
        assert status(lib, call, valid(**kw)) == binding.DSPARK_EINVAL, kw
        assert call in binding.last_error()
    for dt in (binding.DSPARK_F32, 7):
        assert status(lib, call, valid(dtype=dt)) == binding.DSPARK_EDTYPE


@pytest.mark.parametrize("call", CALLS)
def test_nothing_to_do_is_a_no_op(lib, call):
    assert status(lib, call, valid(B=0)) == binding.DSPARK_OK
    assert status(lib, call, valid(rows=0)) == binding.DSPARK_OK


def test_rope_append_refusals(lib):
    f = "dspark_rope_append"
    for kw in (dict(rot_dim=-16), dict(rot_dim=144), dict(rot_dim=24), dict(q=None, k=None, v=None),
               dict(v=None), dict(k=None), dict(row_req=None), dict(packed_pos=None),
               dict(rope_freq=None), dict(q_rot=None), dict(q_stride=8), dict(k_stride=128),
               dict(v_stride=0), dict(k_cache=None), dict(v_cache=None), dict(block_table=None),
               dict(page_size=0), dict(page_size=65537), dict(num_pages=0), dict(max_pages=0),
               dict(max_pages=1 << 30), dict(slot_stride=0), dict(page_stride=-8)):
        assert status(lib, f, valid(**kw)) == binding.DSPARK_EINVAL, kw
    for kw in (dict(q=FAKE + 2), dict(q_rot=FAKE + 8), dict(k=FAKE + 4), dict(v=FAKE + 8),
               dict(k_rot=FAKE + 8), dict(k_cache=FAKE + 8), dict(v_cache=FAKE + 8),
               dict(rope_freq=FAKE + 4), dict(q_stride=12 * 128 + 4), dict(k_stride=12 * 128 + 1),
               dict(v_stride=12 * 128 + 2), dict(head_stride=132), dict(slot_stride=260)):
        assert status(lib, f, valid(**kw)) == binding.DSPARK_EALIGN, kw


@pytest.mark.parametrize("call", CALLS[1:])
def test_attention_refusals(lib, call):
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(q_rot=None), dict(row_off=None), dict(out=None)):
        assert status(lib, call, valid(**kw)) == binding.DSPARK_EINVAL, kw
    for kw in (dict(q_rot=FAKE + 8), dict(out=FAKE + 8)):
        assert status(lib, call, valid(**kw)) == binding.DSPARK_EALIGN, kw
    for kw in (dict(workspace=None), dict(workspace=FAKE + 16), dict(workspace_bytes=8)):
        assert status(lib, call, valid(**kw)) == binding.DSPARK_EWORKSPACE, kw


def test_step_attention_refusals(lib):
    f = "dspark_step_attention"
    for kw in (dict(q_max=66), dict(k_cache=None), dict(v_cache=None), dict(block_table=None),
               dict(page_size=0), dict(num_pages=0), dict(max_pages=0), dict(max_pages=1 << 30)):
        assert status(lib, f, valid(**kw)) == binding.DSPARK_EINVAL, kw
    for kw in (dict(k_cache=FAKE + 8), dict(page_stride=4100)):
        assert status(lib, f, valid(**kw)) == binding.DSPARK_EALIGN, kw


def test_step_attention_refuses_a_wide_group(lib):
    f = "dspark_step_attention"
    size = binding.dspark_attn_workspace_size(256, 1, 128, 9)
    wide = dict(Hq=256, Hkv=1, workspace_bytes=size, head_stride=128)
    assert status(lib, f, valid(**wide)) == binding.DSPARK_EINVAL
    assert "256 query heads" in binding.last_error()


def test_step_attention_refuses_pages_it_cannot_view(lib):
    """Pages whose size has no factor of 8 are gathered: heads and pages must then lie a whole
    number of slots apart, or all heads within one slot."""
    f = "dspark_step_attention"
    for kw in (dict(page_size=12, page_stride=12 * 256 + 128),                    # half a slot over
               dict(page_size=12, slot_stride=128, head_stride=12 * 128 + 64, page_stride=32 * 128)):
        assert status(lib, f, valid(**kw)) == binding.DSPARK_EINVAL, kw
        assert "multiple of 8" in binding.last_error()


def test_step_attention_refuses_a_batch_past_32_bits(lib):
    f = "dspark_step_attention"
    kw = dict(B=65536, rows=65536, max_pages=1 << 20, page_size=64, page_stride=64 * 256)
    assert status(lib, f, valid(**kw)) == binding.DSPARK_EINVAL
    assert "too large a batch" in binding.last_error()


def test_prompt_attention_refusals(lib):
    f = "dspark_prompt_attention"
    for kw in (dict(k_rot=None), dict(v=None), dict(v_stride=128)):
        assert status(lib, f, valid(**kw)) == binding.DSPARK_EINVAL, kw
    for kw in (dict(k_rot=FAKE + 8), dict(v=FAKE + 8), dict(v_stride=12 * 128 + 4)):
        assert status(lib, f, valid(**kw)) == binding.DSPARK_EALIGN, kw


class OnDevice(torch.Tensor):
    """A host tensor that says it is device memory (the binding's checks only)."""
    is_cuda = True


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def buffers():
    h = binding.AttnBuffers.__new__(binding.AttnBuffers)
    h.attn, h._keep = valid(), {}
    return h


def test_binding_checks_what_it_is_given():
    h = buffers()
    with pytest.raises(ValueError, match="CUDA device memory"):
        h.bind(q=torch.zeros((36, 8, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        h.bind(k=fake(36, 2, 128, dtype=torch.float32))
    with pytest.raises(ValueError, match=r"must be \(36, 8, 128\)"):
        h.bind(q=fake(36, 2, 128))
    with pytest.raises(ValueError, match="heads of q must be contiguous"):
        h.bind(q=fake(8, 36, 128).transpose(0, 1))
    with pytest.raises(ValueError, match="q_rot must be contiguous"):
        h.bind(q_rot=fake(36, 9, 128)[:, :8])
    with pytest.raises(ValueError, match="come together"):
        h.bind(k_cache=fake(64, 16, 2, 128))
    with pytest.raises(ValueError, match="same strides"):
        h.bind(k_cache=fake(64, 16, 2, 128), v_cache=fake(64, 2, 16, 128).transpose(1, 2))
    with pytest.raises(ValueError, match="entries of k_cache"):
        h.bind(k_cache=fake(64, 16, 128, 2).transpose(2, 3), v_cache=fake(64, 16, 128, 2).transpose(2, 3))
    with pytest.raises(ValueError, match="row_off must have 5 elements"):
        h.bind(row_off=fake(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="block_table must be int32"):
        h.bind(block_table=fake(4, 8, dtype=torch.int64))


def test_binding_takes_strided_views():
    h = buffers()
    qkv = fake(36, 12 * 128)
    kc, vc = fake(64, 2, 16, 128).transpose(1, 2), fake(64, 2, 16, 128).transpose(1, 2)
    h.bind(q=qkv[:, :1024].unflatten(1, (8, 128)), k=qkv[:, 1024:1280].unflatten(1, (2, 128)),
           k_cache=kc, v_cache=vc)
    a = h.attn
    assert (a.q_stride, a.k_stride) == (12 * 128, 12 * 128)
    assert (a.page_stride, a.slot_stride, a.head_stride) == (4096, 128, 2048)
