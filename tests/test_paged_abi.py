"""Paged cache entry points, host side: layouts, workspace sizes and refusals (CPU).

Every request here is invalid on purpose, or valid on a machine without a GPU (VKV_ERR_CUDA);
none reaches a kernel.
"""
import ctypes
import os

import pytest
import torch

from kv_cache_attention_chunk_b200 import build, vkv

FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    vkv.lib()


def T(ptr=FAKE, sb=64 * 1024, st=1024, sh=128):
    return vkv.vkv_tensor(ptr, sb, st, sh)


def fill(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def map_args(**kw):
    a = vkv.vkv_page_map_args(4, 8, 16, 32, 64, 0)
    for f in ("kv_len", "new_len", "table", "ring", "ring_pos", "kv_len_out", "ring_pos_out", "slot"):
        setattr(a, f, FAKE)
    a.table_stride = 8
    return fill(a, kw)


def append_args(**kw):
    a = vkv.vkv_page_append_args(7, 8, 128, 64, 10, vkv.DTYPE_BF16, vkv.DTYPE_BF16, 0)
    a.k_new, a.v_new = T(sb=0), T(sb=0)
    a.k, a.v = T(), T()
    a.slot = FAKE
    return fill(a, kw)


def select_args(**kw):
    a = vkv.vkv_page_select_args(4, 40, 8, 128, 64, 10, 32, 5, 1, 2, vkv.DTYPE_BF16, 0)
    a.q = T(sb=40 * 128)
    for f in ("kbar", "table", "kv_len", "sel", "workspace"):
        setattr(a, f, FAKE)
    a.table_stride = 32
    a.workspace_bytes = vkv.vkv_page_select_workspace_size(4, 8, 32)
    return fill(a, kw)


def attn_args(**kw):
    a = vkv.vkv_page_attn_args(4, 40, 8, 128, 64, 10, 32, vkv.DTYPE_BF16, vkv.DTYPE_BF16, 0.1, 0, 0, 0, 0)
    a.q, a.o = T(sb=40 * 128), T(sb=40 * 128)
    a.k, a.v = T(), T()
    for f in ("table", "kv_len", "lse", "workspace"):
        setattr(a, f, FAKE)
    a.table_stride = 32
    a.workspace_bytes = 1 << 30
    return fill(a, kw)


CALLS = {"map": (vkv.vkv_page_map, map_args), "append": (vkv.vkv_page_append, append_args),
         "select": (vkv.vkv_page_select, select_args), "attn": (vkv.vkv_page_attn, attn_args)}


def status(which, **kw):
    fn, make = CALLS[which]
    return fn(make(**kw), None)


def test_layouts():
    L = vkv.lib()
    for i, st in ((9, vkv.vkv_page_map_args), (10, vkv.vkv_page_append_args), (11, vkv.vkv_page_select_args),
                  (12, vkv.vkv_page_attn_args)):
        assert L.vkv_abi_sizeof(i) == ctypes.sizeof(st)


@pytest.mark.parametrize("which", list(CALLS))
def test_null_struct_and_no_gpu(which):
    assert getattr(vkv.lib(), f"vkv_page_{which}")(None, None) == 1
    if not torch.cuda.is_available():
        assert status(which) == 6


@pytest.mark.parametrize("kw, want", [
    (dict(R=0), 2), (dict(R=4097), 2), (dict(W=0), 2), (dict(page=0), 2), (dict(n_ring=0), 2), (dict(max_tokens=0), 2),
    (dict(table_stride=7), 2), (dict(R=4096, W=1 << 20, table_stride=1 << 20), 5),
    (dict(W=1 << 20, page=1 << 12, table_stride=1 << 20), 5),
    (dict(kv_len=None), 1), (dict(new_len=None), 1), (dict(table=None), 1), (dict(ring=None), 1),
    (dict(ring_pos=None), 1), (dict(kv_len_out=None), 1), (dict(ring_pos_out=None), 1), (dict(slot=None), 1),
])
def test_map_refusals(kw, want):
    assert status("map", **kw) == want


@pytest.mark.parametrize("kw, want", [
    (dict(d=96), 5), (dict(d=256), 5), (dict(x_dtype=vkv.DTYPE_E4M3), 5), (dict(kv_dtype=vkv.DTYPE_FP16), 5),
    (dict(T=-1), 2), (dict(Hkv=0), 2), (dict(page=0), 2), (dict(n_pages=0), 2), (dict(Hkv=5000), 5),
    (dict(k_scale=FAKE), 5), (dict(v_scale=FAKE), 5), (dict(k=T(ptr=0)), 1), (dict(slot=None), 1),
    (dict(k_new=T(ptr=0)), 1), (dict(k=T(ptr=FAKE + 8)), 3), (dict(v=T(st=1028)), 3), (dict(v_new=T(sh=132)), 3),
    (dict(kv_dtype=vkv.DTYPE_E4M3, k=T(st=1032)), 3), (dict(kbar=FAKE + 8), 3),
])
def test_append_refusals(kw, want):
    assert status("append", **kw) == want


@pytest.mark.parametrize("kw, want", [
    (dict(d=32), 5), (dict(q_dtype=vkv.DTYPE_E4M3), 5), (dict(H=41), 2), (dict(R=0), 2), (dict(R=4097), 2),
    (dict(topk=0), 2), (dict(topk=4097), 2), (dict(topk=2), 2), (dict(sink_pages=-1), 2), (dict(table_stride=31), 2),
    (dict(W=0), 2), (dict(n_pages=0), 2), (dict(q=T(ptr=0)), 1), (dict(kbar=None), 1), (dict(sel=None), 1),
    (dict(q=T(ptr=FAKE + 4)), 3), (dict(kbar=FAKE + 4), 3), (dict(workspace=None), 7), (dict(workspace_bytes=64), 7),
    (dict(workspace=FAKE + 16), 3), (dict(page=1 << 30), 5),
])
def test_select_refusals(kw, want):
    assert status("select", **kw) == want


@pytest.mark.parametrize("kw, want", [
    (dict(d=96), 5), (dict(q_dtype=vkv.DTYPE_E4M3), 5), (dict(kv_dtype=vkv.DTYPE_FP16), 5), (dict(H=41), 2),
    (dict(R=0), 2), (dict(R=4097), 2), (dict(sink=-1), 2), (dict(window=-1), 2), (dict(scale=0.0), 2),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(topk=3), 2), (dict(sel=FAKE), 2),
    (dict(sel=FAKE, topk=3, window=5), 2), (dict(k_scale=FAKE), 5), (dict(table_stride=31), 2), (dict(page=1 << 30), 5),
    (dict(q=T(ptr=0)), 1), (dict(lse=None), 1), (dict(o=T(ptr=FAKE + 2)), 3), (dict(k=T(sb=1028)), 3),
    (dict(H=8192), 5),
])
def test_attn_refusals(kw, want):
    assert status("attn", **kw) == want


def test_binding_of_another_torch_is_rebuilt_and_never_loaded(monkeypatch):
    assert build.binding_fits()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not build.binding_fits()
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        raise FileNotFoundError("not run")

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(FileNotFoundError):  # though no file is newer than it
        build.build()
    assert any(str(x).endswith("vkv_binding.cpp") for x in commands[0])
    monkeypatch.setattr(vkv, "_binding", None)
    with pytest.raises(RuntimeError, match="another torch"):
        vkv._page_binding()


def test_append_refuses_pages_whose_rows_could_overflow():
    """The mean's loop over a page's earlier rows steps up to 64 rows past the last, in 32 bits."""
    for page in (2**31 - 1, 2**31 - 64, 2**30 + 1):
        assert status("append", page=page) == 5, page
    if not torch.cuda.is_available():  # the longest that is taken
        assert status("append", page=2**30) == 6


def test_select_refuses_tables_whose_columns_could_overflow():
    """The score kernel's column numbers run up to 64 past the table's width, in 32 bits."""
    wide = dict(R=1, page=1, topk=5, workspace_bytes=1 << 62)
    for W in (2**31 - 1, 2**31 - 64, 2**31 - 256):
        assert status("select", W=W, table_stride=W, **wide) == 5, W
    if not torch.cuda.is_available():  # the widest that is taken
        assert status("select", W=2**31 - 257, table_stride=2**31, **wide) == 6


def test_wrapper_refusals():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):  # not on a GPU
        vkv.page_map(i32(2), i32(2), i32(2, 3), i32(4), torch.zeros(2, dtype=torch.int64), 16, 8)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        vkv.page_attn(q, c, c, i32(2, 3), i32(2))
    with pytest.raises(ValueError):  # another d
        vkv.page_attn(q[:, :, :32], c, c, i32(2, 3), i32(2))
    with pytest.raises(ValueError):  # k and v differ
        vkv.page_attn(q, c, c[:2], i32(2, 3), i32(2))
    with pytest.raises(ValueError):
        vkv.page_append(c[0], c[0, :8], torch.zeros(16, dtype=torch.int64), c, c)
    with pytest.raises(ValueError):
        vkv.page_select(q, torch.zeros(3, 2, 32), i32(2, 3), i32(2), 16, 2)


def test_workspace_sizes():
    assert vkv.vkv_page_select_workspace_size(0, 1, 1) == 0
    assert vkv.vkv_page_select_workspace_size(3, 8, 100) >= 3 * 8 * 100 * 8
    assert vkv.vkv_page_attn_workspace_size(7, 2, 128) == 0
    assert vkv.vkv_page_attn_workspace_size(8, 2, 96) == 0


def test_kernels_launched_ahead_load_coherently():
    """Read-only-path loads are for memory that nobody writes while the kernel is resident: a kernel that
    takes its place while the stream's last one still runs has none."""
    for name in ("vkv_page.cuh", "vkv_page_map.cu", "vkv_page_append.cu", "vkv_page_select.cu", "vkv_page_attn.cu"):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        for word in ("__ldg", "global.nc", "__restrict__"):
            assert word not in text, (name, word)
