"""The C ABI of reading less of a long cache without a GPU: symbols, sizes and every refusal before a launch."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import long_reference as G
from bit_quantized_decode_amd import binding as B
from test_attn_abi_cpu import A, BAD_CACHES, L, ODD, attn, desc  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_attn_long.h")
BIG = 1 << 40


def test_every_declared_symbol_is_exported(L):  # noqa: F811
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(nvfp4_\w+)\s*\(", text))
    assert names == set(B.EXPORTED_ATTN_LONG)
    for name in names:
        assert hasattr(L, name), name
    assert f"#define NVFP4_SELECT_COUNTER_BYTES {B.NVFP4_SELECT_COUNTER_BYTES}" in text


def shared(d, own=(), **over):
    a = B.AttnSharedArgs(attn=attn(d, **dict(own)), prefix_table=A, prefix_width=100, prefix_len=A)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def weigh(d, own=(), **over):
    a = B.AttnWeighArgs(attn=attn(d, **dict(own)), weights=A, decay=0.5, weights_out=A)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def select(d, **over):
    a = B.KvSelectArgs(cache=ctypes.pointer(d), batch=4, q_heads=40, q=A, ldq=5120, bounds=A, page_table=A, table_width=500,
                       seq_lens=A, budget=16, pages_out=A, lens_out=A, workspace=A, workspace_bytes=BIG)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def evict(**over):
    a = B.KvEvictArgs(batch=4, kv_heads=8, page_size=64, weights=A, page_table=A, table_width=9000, seq_lens=A, budget=16, sink=1,
                      recent=2, table_out=A, lens_out=A, weights_out=A, freed=A, workspace=A, workspace_bytes=BIG)
    for k, v in over.items():
        setattr(a, k, v)
    return a


ATTN = [
    (dict(batch=-1), B.NVFP4_ERR_SHAPE), (dict(batch=65537), B.NVFP4_ERR_SHAPE), (dict(q_heads=12), B.NVFP4_ERR_SHAPE),
    (dict(table_width=-1), B.NVFP4_ERR_SHAPE), (dict(batch=65536, table_width=1 << 22), B.NVFP4_ERR_SHAPE),
    (dict(window=-1), B.NVFP4_ERR_ARG), (dict(scale=0.0), B.NVFP4_ERR_ARG), (dict(scale=float("inf")), B.NVFP4_ERR_ARG),
    (dict(ldq=5112), B.NVFP4_ERR_SHAPE), (dict(ldo=5124), B.NVFP4_ERR_SHAPE), (dict(q=None), B.NVFP4_ERR_NULL),
    (dict(out=None), B.NVFP4_ERR_NULL), (dict(seq_lens=None), B.NVFP4_ERR_NULL), (dict(page_table=None), B.NVFP4_ERR_NULL),
    (dict(q=A + 8), B.NVFP4_ERR_ALIGN), (dict(lse=ODD), B.NVFP4_ERR_ALIGN), (dict(workspace=None), B.NVFP4_ERR_WORKSPACE),
    (dict(workspace_bytes=1024), B.NVFP4_ERR_WORKSPACE), (dict(workspace=A + 8), B.NVFP4_ERR_ALIGN),
    (dict(batch=0, q=None, out=None, workspace=None), B.NVFP4_OK)]


@pytest.mark.parametrize("own,status", ATTN)
def test_refusals_that_all_attention_shares(L, own, status):  # noqa: F811
    d = desc()
    assert L.nvfp4_attn_decode_heads(ctypes.byref(attn(d, **own)), None) == status
    assert L.nvfp4_attn_weigh(ctypes.byref(weigh(d, own)), None) == status
    if own.get("window", 0) == 0:
        assert L.nvfp4_attn_shared(ctypes.byref(shared(d, own)), None) == status


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_cache_refusals(L, over, status):  # noqa: F811
    d, n = desc(**over), ctypes.c_size_t()
    assert L.nvfp4_attn_decode_heads(ctypes.byref(attn(d)), None) == status
    assert L.nvfp4_kv_bounds(ctypes.byref(d), A, 4, A, None) == status
    for make, name in ((shared, "attn_shared"), (weigh, "attn_weigh"), (select, "kv_select")):
        a = make(d)
        assert getattr(L, f"nvfp4_{name}")(ctypes.byref(a), None) == status
        assert getattr(L, f"nvfp4_{name}_workspace_bytes")(ctypes.byref(a), ctypes.byref(n)) == status


@pytest.mark.parametrize("own,over,status", [
    ({}, dict(prefix_width=-1), B.NVFP4_ERR_SHAPE), ({}, dict(prefix_width=(1 << 24) + 1), B.NVFP4_ERR_SHAPE),
    (dict(window=1), {}, B.NVFP4_ERR_ARG), ({}, dict(prefix_table=None), B.NVFP4_ERR_NULL),
    ({}, dict(prefix_len=None), B.NVFP4_ERR_NULL), ({}, dict(prefix_table=ODD), B.NVFP4_ERR_ALIGN),
    ({}, dict(prefix_len=ODD), B.NVFP4_ERR_ALIGN),
    (dict(batch=65536, q_heads=16392, ldq=1 << 22, ldo=1 << 22, table_width=0), dict(prefix_width=1), B.NVFP4_ERR_SHAPE),
    (dict(batch=4096, table_width=1), dict(prefix_width=1 << 24), B.NVFP4_ERR_SHAPE),
    (dict(batch=0, workspace=None), dict(prefix_table=None, prefix_len=None), B.NVFP4_OK),
    (dict(workspace=None), dict(prefix_width=0, prefix_table=None), B.NVFP4_ERR_WORKSPACE)])
def test_shared_refusals(L, own, over, status):  # noqa: F811
    d = desc()
    assert L.nvfp4_attn_shared(ctypes.byref(shared(d, own, **over)), None) == status


@pytest.mark.parametrize("own,over,status", [
    ({}, dict(decay=-0.5), B.NVFP4_ERR_ARG), ({}, dict(decay=float("nan")), B.NVFP4_ERR_ARG),
    ({}, dict(decay=float("inf")), B.NVFP4_ERR_ARG), ({}, dict(weights=None), B.NVFP4_ERR_NULL),
    ({}, dict(weights_out=None), B.NVFP4_ERR_NULL), ({}, dict(weights=ODD), B.NVFP4_ERR_ALIGN),
    ({}, dict(weights_out=ODD), B.NVFP4_ERR_ALIGN),
    (dict(batch=65536, table_width=4097, window=16), {}, B.NVFP4_ERR_SHAPE),
    (dict(workspace=None), dict(weights=None, decay=0.0), B.NVFP4_ERR_WORKSPACE),
    (dict(workspace=None, table_width=0), dict(weights=None, weights_out=None), B.NVFP4_ERR_WORKSPACE)])
def test_weigh_refusals(L, own, over, status):  # noqa: F811
    d = desc()
    assert L.nvfp4_attn_weigh(ctypes.byref(weigh(d, own, **over)), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), B.NVFP4_ERR_SHAPE), (dict(batch=65537), B.NVFP4_ERR_SHAPE), (dict(q_heads=12), B.NVFP4_ERR_SHAPE),
    (dict(q_heads=0), B.NVFP4_ERR_SHAPE), (dict(q_heads=32776), B.NVFP4_ERR_SHAPE), (dict(table_width=-1), B.NVFP4_ERR_SHAPE),
    (dict(table_width=(1 << 24) + 1), B.NVFP4_ERR_SHAPE), (dict(budget=0), B.NVFP4_ERR_SHAPE), (dict(budget=-3), B.NVFP4_ERR_SHAPE),
    (dict(budget=(1 << 24) + 1), B.NVFP4_ERR_SHAPE), (dict(ldq=5112), B.NVFP4_ERR_SHAPE), (dict(ldq=5124), B.NVFP4_ERR_SHAPE),
    (dict(q=None), B.NVFP4_ERR_NULL), (dict(bounds=None), B.NVFP4_ERR_NULL), (dict(page_table=None), B.NVFP4_ERR_NULL),
    (dict(seq_lens=None), B.NVFP4_ERR_NULL), (dict(pages_out=None), B.NVFP4_ERR_NULL), (dict(lens_out=None), B.NVFP4_ERR_NULL),
    (dict(q=A + 8), B.NVFP4_ERR_ALIGN), (dict(bounds=A + 8), B.NVFP4_ERR_ALIGN), (dict(page_table=ODD), B.NVFP4_ERR_ALIGN),
    (dict(seq_lens=ODD), B.NVFP4_ERR_ALIGN), (dict(pages_out=ODD), B.NVFP4_ERR_ALIGN), (dict(lens_out=ODD), B.NVFP4_ERR_ALIGN),
    (dict(workspace=None), B.NVFP4_ERR_WORKSPACE), (dict(workspace_bytes=4096), B.NVFP4_ERR_WORKSPACE),
    (dict(workspace=A + 8), B.NVFP4_ERR_ALIGN), (dict(batch=0, q=None, workspace=None), B.NVFP4_OK)])
def test_select_refusals(L, over, status):  # noqa: F811
    d = desc(pool=None)
    assert L.nvfp4_kv_select(ctypes.byref(select(d, **over)), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), B.NVFP4_ERR_SHAPE), (dict(batch=65537), B.NVFP4_ERR_SHAPE), (dict(kv_heads=0), B.NVFP4_ERR_SHAPE),
    (dict(kv_heads=1025), B.NVFP4_ERR_SHAPE), (dict(page_size=8), B.NVFP4_ERR_SHAPE), (dict(page_size=40), B.NVFP4_ERR_SHAPE),
    (dict(page_size=1 << 17), B.NVFP4_ERR_SHAPE), (dict(table_width=-1), B.NVFP4_ERR_SHAPE),
    (dict(table_width=(1 << 24) + 1), B.NVFP4_ERR_SHAPE), (dict(budget=0), B.NVFP4_ERR_SHAPE),
    (dict(budget=(1 << 24) + 1), B.NVFP4_ERR_SHAPE), (dict(sink=-1), B.NVFP4_ERR_ARG), (dict(recent=0), B.NVFP4_ERR_ARG),
    (dict(weights=None), B.NVFP4_ERR_NULL), (dict(page_table=None), B.NVFP4_ERR_NULL), (dict(seq_lens=None), B.NVFP4_ERR_NULL),
    (dict(table_out=None), B.NVFP4_ERR_NULL), (dict(lens_out=None), B.NVFP4_ERR_NULL), (dict(weights=ODD), B.NVFP4_ERR_ALIGN),
    (dict(page_table=ODD), B.NVFP4_ERR_ALIGN), (dict(seq_lens=ODD), B.NVFP4_ERR_ALIGN), (dict(table_out=ODD), B.NVFP4_ERR_ALIGN),
    (dict(lens_out=ODD), B.NVFP4_ERR_ALIGN), (dict(weights_out=ODD), B.NVFP4_ERR_ALIGN), (dict(freed=ODD), B.NVFP4_ERR_ALIGN),
    (dict(workspace=None), B.NVFP4_ERR_WORKSPACE), (dict(workspace_bytes=100), B.NVFP4_ERR_WORKSPACE),
    (dict(workspace=A + 8), B.NVFP4_ERR_ALIGN), (dict(batch=0, weights=None, table_out=None, workspace=None), B.NVFP4_OK)])
def test_evict_refusals(L, over, status):  # noqa: F811
    assert L.nvfp4_kv_evict(ctypes.byref(evict(**over)), None) == status


def test_bounds_refusals(L):  # noqa: F811
    d = desc()
    call = lambda c=d, pages=A, n=4, bounds=A: L.nvfp4_kv_bounds(ctypes.byref(c), pages, n, bounds, None)  # noqa: E731
    assert call(n=-1) == call(n=(1 << 24) + 1) == B.NVFP4_ERR_SHAPE
    assert call(c=desc(pages=1, kv_heads=1024), n=(1 << 22) + 1) == B.NVFP4_ERR_SHAPE
    assert call(pages=None) == call(bounds=None) == call(c=desc(pool=None)) == B.NVFP4_ERR_NULL
    assert call(pages=ODD) == call(bounds=A + 8) == call(c=desc(pool=A + 8)) == B.NVFP4_ERR_ALIGN
    assert call(n=0, pages=None, bounds=None) == call(n=0, c=desc(pool=None)) == B.NVFP4_OK
    assert L.nvfp4_kv_bounds(None, A, 4, A, None) == B.NVFP4_ERR_NULL


def test_null_arguments(L):  # noqa: F811
    n = ctypes.c_size_t()
    for name, make in (("attn_shared", shared), ("attn_weigh", weigh), ("kv_select", select), ("kv_evict", lambda d: evict())):
        assert getattr(L, f"nvfp4_{name}")(None, None) == B.NVFP4_ERR_NULL
        assert getattr(L, f"nvfp4_{name}_workspace_bytes")(None, ctypes.byref(n)) == B.NVFP4_ERR_NULL
        d = desc()
        assert getattr(L, f"nvfp4_{name}_workspace_bytes")(ctypes.byref(make(d)), None) == B.NVFP4_ERR_NULL
    for args, name in ((B.AttnSharedArgs(), "attn_shared"), (B.AttnWeighArgs(), "attn_weigh"), (B.KvSelectArgs(), "kv_select")):
        assert getattr(L, f"nvfp4_{name}")(ctypes.byref(args), None) == B.NVFP4_ERR_NULL
    assert L.nvfp4_attn_decode_heads(None, None) == B.NVFP4_ERR_NULL


def test_workspaces(L):  # noqa: F811
    """Sizes depend on what the header says and are what the calls ask for; at the largest shapes they do not wrap."""
    def need(name, a):
        n = ctypes.c_size_t()
        assert getattr(L, f"nvfp4_{name}_workspace_bytes")(ctypes.byref(a), ctypes.byref(n)) == B.NVFP4_OK
        return n.value

    d = desc()
    plain = need("attn_decode", attn(d))
    blank = dict(q=None, out=None, page_table=None, seq_lens=None, workspace=None, scale=0.0, ldq=0, ldo=0)
    s = need("attn_shared", shared(d, blank, prefix_table=None, prefix_len=None, prefix_width=1 << 16))
    assert s > plain and need("attn_shared", shared(d, prefix_width=0)) == plain
    # A prefix that each sequence reads by itself is so much more of its table; to the largest tables it is not.
    assert need("attn_shared", shared(d)) == need("attn_decode", attn(d, table_width=attn(d).table_width + 100))
    most = (1 << 30) // d.page_size
    assert need("attn_shared", shared(d, dict(batch=1, q_heads=8, table_width=most), prefix_width=most)) > plain
    w = need("attn_weigh", weigh(d, blank, weights=None, weights_out=None, decay=-1.0))
    assert w > plain + 4 * 4 * 40 * 16
    for name, a, n in (("attn_shared", shared(d, dict(workspace_bytes=s - 1), prefix_width=1 << 16), s), ("attn_weigh", weigh(d, dict(workspace_bytes=w - 1)), w)):
        assert getattr(L, f"nvfp4_{name}")(ctypes.byref(a), None) == B.NVFP4_ERR_WORKSPACE
        assert str(n).encode() in L.nvfp4_last_error()
    for name, a in (("attn_shared", shared(d, dict(batch=0))), ("attn_weigh", weigh(d, dict(batch=0))), ("kv_select", select(d, batch=0)),
                    ("kv_evict", evict(batch=0)), ("kv_select", select(d, budget=500)), ("kv_evict", evict(table_width=4096))):
        assert need(name, a) == 0, name
    # One workgroup a (sequence, kv head), whose keys fit LDS, needs none.
    assert need("kv_select", select(d, batch=128)) == 0 and need("kv_select", select(d)) == 4096 + 4 * 8 * 500 * 8
    assert need("kv_select", select(d, batch=128, table_width=4097)) == 4096 + 128 * 8 * 4097 * 8
    assert need("kv_evict", evict()) == 4 * 9000 * 8
    wide = desc(kv_heads=1, page_size=16, pages=1 << 20)
    assert need("kv_evict", evict(batch=65536, page_size=16, table_width=1 << 26)) == 1 << 45
    assert need("kv_select", select(wide, batch=65536, q_heads=1, table_width=1 << 26, budget=1)) == 4096 + (1 << 45)
    # Under a window the kept sums are those of the window.
    assert need("attn_weigh", weigh(wide, dict(q_heads=1, table_width=1 << 24, window=100))) < 1 << 24


def test_binding_refuses_host_tensors_and_wrong_shapes():
    cache = B.KvCache(4, 16, 1, 64, B.NVFP4_KV_BF16, device="cpu")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, w = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 1, 3)
    bounds = torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: B.attn_shared(q, cache, i32(1), i32(1), i32(2, 3), i32(2)), lambda: B.kv_bounds(cache, i32(2)),
                 lambda: B.kv_select(q, cache, bounds, i32(2, 3), i32(2), 2), lambda: B.attn_weigh(q, cache, i32(2, 3), i32(2), w),
                 lambda: B.kv_evict(w, i32(2, 3), i32(2), 16, 2), lambda: B.attn_decode(q, cache, i32(2, 1, 3), i32(2))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for prepared in (B.attn_shared_prepared, B.attn_shared):
        with pytest.raises(ValueError, match="prefix_pages"):
            prepared(q, cache, i32(1, 1), i32(1), i32(2, 3), i32(2))
    for prepared in (B.attn_weigh_prepared, B.attn_weigh):
        with pytest.raises(ValueError, match="decay"):
            prepared(q, cache, i32(2, 3), i32(2), None)
        with pytest.raises(ValueError, match="decay"):
            prepared(q, cache, i32(2, 3), i32(2), None, 0.0)
    with pytest.raises(ValueError, match="weights"):
        B.kv_evict(w[0], i32(2, 3), i32(2), 16, 2)
    with pytest.raises(ValueError, match="page_table"):
        B.kv_select(q, cache, bounds, i32(2, 1, 3), i32(2), 2)
    with pytest.raises(ValueError, match="pages"):
        B.kv_bounds(cache, i32(2, 2))
    with pytest.raises(ValueError, match="contiguous"):
        B.kv_select(q, cache, bounds, i32(2, 3), i32(2), 2, ws=torch.zeros(1, dtype=torch.uint8).expand(100))


# ---- the tests' own reference ---------------------------------------------------

def test_reference_selection():
    """A hand-made case: two heads that rank differently, ties, a page that is gone, a short sequence."""
    q = torch.zeros(2, 2, 16, dtype=torch.bfloat16)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    bounds = np.zeros((6, 2, 2, 16))
    for p, (lo, hi) in enumerate([(0, 1), (-3, 2), (-1, 2), (0, 0), (9, 9), (-9, 9)]):
        bounds[p, :, 0, 0], bounds[p, :, 1, 0] = lo, hi
    table = np.array([[0, 1, 2, 3, -1, 4], [5, 0, 1, 2, 3, 4]])
    pages, lens = G.selection(q, bounds, table, [6 * 16 - 2, 10], 3, 16, 6)
    assert pages[0].tolist() == [[1, 2, 4], [1, 2, 4]] and pages[1].tolist() == [[5, -1, -1]] * 2
    assert lens.tolist() == [2 * 16 + 14, 10]
    pages, _ = G.selection(q, bounds, table, [96, 0], 2, 16, 6)
    assert pages[0].tolist() == [[1, 4], [1, 4]] and (pages[1] == -1).all()


def test_reference_eviction():
    weights = np.array([[[1, 5, 2, 5, 0, 3, 0.5], [0, 0, 2, 0, 0, 0, 0]]], np.float32)
    table = np.array([[10, 11, 12, 13, -1, 15, 16]])
    for budget, sink, recent, want in [(7, 0, 1, [10, 11, 12, 13, 15, 16]), (1, 0, 1, [16]), (2, 0, 1, [11, 16]), (3, 0, 1, [11, 13, 16]),
                                       (3, 1, 1, [10, 11, 16]), (2, 1, 5, [15, 16]), (4, 2, 2, [10, 11, 15, 16]), (5, 0, 4, [11, 12, 13, 15, 16])]:
        out, lens, freed, moved = G.eviction(weights, table, [7 * 16 - 1], 16, budget, sink, recent)
        assert out[0][out[0] >= 0].tolist() == want, (budget, sink, recent)
        assert lens[0] == len(want) * 16 - 1
        assert sorted(freed[0][freed[0] >= 0].tolist() + want) == [10, 11, 12, 13, 15, 16]
        assert moved[0, 0, :len(want)].tolist() == [float(weights[0, 0, p - 10]) for p in want]
