"""The attention side's C ABI without a GPU: symbols, sizes, the frequency table, and every refusal before a launch."""
import ctypes
import math
import os
import re
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_attn.h")
A = 0x10000       # placeholders: never dereferenced on these paths
ODD = A + 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        from bit_quantized_decode_amd import build
        build.build()
    return B.lib()


def test_every_declared_symbol_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(nvfp4_\w+)\s*\(", text))
    assert names == set(B.EXPORTED_ATTN)
    for name in names:
        assert hasattr(L, name), name


# ---- the frequency table ------------------------------------------------------

def exact_freqs(rot, base, scaling=None):
    """f_i in turns per position, to 50 digits."""
    getcontext().prec = 50
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582")
    b = Decimal(base)
    f = [(-(Decimal(2 * i) / rot) * b.ln()).exp() / (2 * pi) for i in range(rot // 2)]
    if scaling is None:
        return f
    if scaling[0] == "linear":
        return [x / Decimal(scaling[1]) for x in f]
    factor, trained, fast, slow = (list(scaling[1:]) + [32.0, 1.0])[:4] if len(scaling) == 3 else scaling[1:]

    def pair(turns):
        return Decimal(rot) * (Decimal(trained) / (Decimal(turns) * 2 * pi)).ln() / (2 * b.ln())
    low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    out = []
    for i, x in enumerate(f):
        ramp = min(max(Decimal(i - low) / max(Decimal(high - low), Decimal("0.001")), Decimal(0)), Decimal(1))
        out.append(x * (1 - ramp) + x / Decimal(factor) * ramp)
    return out


@pytest.mark.parametrize("rot,base,scaling", [
    (128, 1e4, None), (16, 1e6, None), (256, 5e5, None), (64, 1e4, ("linear", 4.0)), (128, 1e6, ("yarn", 8.0, 32768)),
    (96, 1e4, ("yarn", 64.0, 4096, 32.0, 1.0)), (64, 1e4, ("yarn", 1.0, 4096)), (48, 2.0, ("yarn", 4.0, 7, 3.0, 0.5))])
def test_frequencies(rot, base, scaling):
    freqs, magnitude = B.rope_freqs(rot, base, scaling)
    got = [int(f) % 2 ** 64 for f in freqs.tolist()]
    for g, f in zip(got, exact_freqs(rot, base, scaling)):
        # Extended precision (2^-64) of the exponent, at most 14, and of a few operations.
        assert abs(Decimal(g) - f * 2 ** 64) <= f * 2 ** 64 * Decimal(2) ** -58 + 1
    factor = scaling[1] if scaling and scaling[0] == "yarn" else 1.0
    assert magnitude == np.float32(0.1 * math.log(factor) + 1.0)


def test_frequency_refusals():
    for rot, base, scaling, status in [
            (8, 1e4, None, B.NVFP4_ERR_SHAPE), (272, 1e4, None, B.NVFP4_ERR_SHAPE), (-16, 1e4, None, B.NVFP4_ERR_SHAPE),
            (64, 1.0, None, B.NVFP4_ERR_ARG), (64, float("nan"), None, B.NVFP4_ERR_ARG),
            (64, float("inf"), None, B.NVFP4_ERR_ARG), (64, 1e4, ("linear", 0.5), B.NVFP4_ERR_ARG),
            (64, 1e4, ("yarn", 2.0, 0.0), B.NVFP4_ERR_ARG), (64, 1e4, ("yarn", 2.0, 100, 1.0, 1.0), B.NVFP4_ERR_ARG),
            (64, 1e4, ("yarn", 2.0, 100, 32.0, -1.0), B.NVFP4_ERR_ARG)]:
        with pytest.raises(B.Nvfp4Error) as e:
            B.rope_freqs(rot, base, scaling)
        assert e.value.status == status, (rot, base, scaling)
    for scaling in (("yarn", 2.0), ("linear",), ("cubic", 2.0), ("linear", 2.0, 3.0), ("yarn", 2.0, 100, 32.0)):
        with pytest.raises(ValueError):
            B.rope_freqs(64, 1e4, scaling)
    with pytest.raises(ValueError):
        B.rope_table(64, layout="diagonal", device="cpu")
    c, m = B.RopeConfig(rot_dim=64, base=1e4, scaling=7), ctypes.c_float()
    f = (ctypes.c_uint64 * 32)()
    assert B.lib().nvfp4_rope_freqs(ctypes.byref(c), f, ctypes.byref(m)) == B.NVFP4_ERR_ARG
    assert B.lib().nvfp4_rope_freqs(ctypes.byref(c), None, ctypes.byref(m)) == B.NVFP4_ERR_NULL
    assert B.lib().nvfp4_rope_freqs(None, f, ctypes.byref(m)) == B.NVFP4_ERR_NULL


# ---- refusals -----------------------------------------------------------------

def desc(**over):
    d = dict(pool=A, pages=8, page_size=64, kv_heads=8, head_dim=128, format=B.NVFP4_KV_NVFP4, k_scale=1.0, v_scale=1.0)
    return B.KvCacheDesc(**(d | over))


BAD_CACHES = [
    (dict(format=3), B.NVFP4_ERR_DTYPE), (dict(head_dim=0), B.NVFP4_ERR_SHAPE), (dict(head_dim=120), B.NVFP4_ERR_SHAPE),
    (dict(head_dim=272), B.NVFP4_ERR_SHAPE), (dict(page_size=8), B.NVFP4_ERR_SHAPE), (dict(page_size=24), B.NVFP4_ERR_SHAPE),
    (dict(page_size=1 << 17), B.NVFP4_ERR_SHAPE), (dict(kv_heads=0), B.NVFP4_ERR_SHAPE), (dict(kv_heads=1025), B.NVFP4_ERR_SHAPE),
    (dict(pages=0), B.NVFP4_ERR_SHAPE), (dict(pages=1 << 40), B.NVFP4_ERR_SHAPE), (dict(pages=(1 << 34) // 512 + 1), B.NVFP4_ERR_SHAPE),
    (dict(k_scale=0.0), B.NVFP4_ERR_ARG), (dict(v_scale=float("inf")), B.NVFP4_ERR_ARG), (dict(k_scale=float("nan")), B.NVFP4_ERR_ARG),
    (dict(k_scale=-1.0), B.NVFP4_ERR_ARG), (dict(v_scale=1e-30), B.NVFP4_ERR_ARG),
    (dict(format=B.NVFP4_KV_BF16, k_scale=0.5), B.NVFP4_ERR_ARG), (dict(format=B.NVFP4_KV_E4M3, v_scale=2.0), B.NVFP4_ERR_ARG),
]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_cache_refusals(L, over, status):
    d, n = desc(**over), ctypes.c_size_t()
    assert L.nvfp4_kv_cache_bytes(ctypes.byref(d), ctypes.byref(n)) == status
    a = append(d)
    assert L.nvfp4_kv_append(ctypes.byref(a), None) == status
    assert L.nvfp4_kv_read(ctypes.byref(d), A, 4, A, 1024, A, 1024, B.NVFP4_BF16, None) == status
    t = attn(d)
    assert L.nvfp4_attn_decode(ctypes.byref(t), None) == status
    assert L.nvfp4_attn_decode_workspace_bytes(ctypes.byref(t), ctypes.byref(n)) == status


def test_cache_bytes(L):
    for fmt, db, group in [(0, 1, 4096), (0, 2, 8192), (1, 2, 4096 + 32), (1, 4, 8192 + 32), (2, 1, 1024 + 128),
                           (2, 2, 2048 + 256), (2, 3, 3 * 1024 + 256 + 192), (2, 4, 4096 + 512)]:
        for d in (64 * db, 64 * db - 48):
            n = ctypes.c_size_t()
            c = desc(format=fmt, head_dim=d, pages=7, page_size=48, kv_heads=3, pool=None)
            assert L.nvfp4_kv_cache_bytes(ctypes.byref(c), ctypes.byref(n)) == 0
            assert n.value == 7 * 3 * 3 * group
    assert L.nvfp4_kv_cache_bytes(ctypes.byref(desc()), None) == B.NVFP4_ERR_NULL
    assert L.nvfp4_kv_cache_bytes(None, ctypes.byref(ctypes.c_size_t())) == B.NVFP4_ERR_NULL
    with pytest.raises(ValueError):
        B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device="cpu", pool=torch.empty(100, dtype=torch.uint8))


def rope(**over):
    a = B.RopeArgs(tokens=4, heads=2, head_dim=64, rot_dim=64, magnitude=1.0, positions=A, freqs=A, x=A, x_dtype=1, ldx=128,
                   y=2 * A, y_dtype=1, ldy=128)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), B.NVFP4_ERR_SHAPE), (dict(tokens=(1 << 24) + 1), B.NVFP4_ERR_SHAPE), (dict(heads=-1), B.NVFP4_ERR_SHAPE),
    (dict(heads=32769), B.NVFP4_ERR_SHAPE), (dict(head_dim=60), B.NVFP4_ERR_SHAPE), (dict(rot_dim=80), B.NVFP4_ERR_SHAPE),
    (dict(rot_dim=40), B.NVFP4_ERR_SHAPE), (dict(rot_dim=-16), B.NVFP4_ERR_SHAPE), (dict(layout=2), B.NVFP4_ERR_ARG),
    (dict(magnitude=float("nan")), B.NVFP4_ERR_ARG), (dict(x_dtype=2), B.NVFP4_ERR_DTYPE), (dict(y_dtype=-1), B.NVFP4_ERR_DTYPE),
    (dict(ldx=120), B.NVFP4_ERR_SHAPE), (dict(ldx=132), B.NVFP4_ERR_SHAPE), (dict(ldy=64), B.NVFP4_ERR_SHAPE),
    (dict(x=None), B.NVFP4_ERR_NULL), (dict(y=None), B.NVFP4_ERR_NULL), (dict(positions=None), B.NVFP4_ERR_NULL),
    (dict(freqs=None), B.NVFP4_ERR_NULL), (dict(x=A + 8), B.NVFP4_ERR_ALIGN), (dict(y=A + 8), B.NVFP4_ERR_ALIGN),
    (dict(positions=ODD), B.NVFP4_ERR_ALIGN), (dict(freqs=A + 4), B.NVFP4_ERR_ALIGN), (dict(y=A, ldy=256), B.NVFP4_ERR_ARG),
    (dict(y=A, y_dtype=0), B.NVFP4_ERR_ARG), (dict(tokens=0, x=None), B.NVFP4_OK), (dict(heads=0, y=None), B.NVFP4_OK)])
def test_rope_refusals(L, over, status):
    assert L.nvfp4_rope(ctypes.byref(rope(**over)), None) == status


def append(d, **over):
    a = B.KvAppendArgs(cache=ctypes.pointer(d), tokens=4, slots=A, k=A, v=A, dtype=1, ldk=1024, ldv=1024, freqs=A, positions=A,
                       rot_dim=64, magnitude=1.0, q_heads=16, q=A, ldq=2048, q_out=2 * A, ldqo=2048)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), B.NVFP4_ERR_SHAPE), (dict(tokens=1 << 25), B.NVFP4_ERR_SHAPE), (dict(dtype=3), B.NVFP4_ERR_DTYPE),
    (dict(ldk=1016), B.NVFP4_ERR_SHAPE), (dict(ldv=1028), B.NVFP4_ERR_SHAPE), (dict(ldq=1024), B.NVFP4_ERR_SHAPE),
    (dict(ldqo=2044), B.NVFP4_ERR_SHAPE), (dict(rot_dim=144), B.NVFP4_ERR_SHAPE), (dict(layout=-1), B.NVFP4_ERR_ARG),
    (dict(magnitude=float("inf")), B.NVFP4_ERR_ARG), (dict(freqs=None), B.NVFP4_ERR_ARG), (dict(q_heads=0), B.NVFP4_ERR_SHAPE),
    (dict(q_heads=1 << 16), B.NVFP4_ERR_SHAPE), (dict(slots=None), B.NVFP4_ERR_NULL), (dict(k=None), B.NVFP4_ERR_NULL),
    (dict(v=None), B.NVFP4_ERR_NULL), (dict(q_out=None), B.NVFP4_ERR_NULL), (dict(positions=None), B.NVFP4_ERR_NULL),
    (dict(slots=A + 4), B.NVFP4_ERR_ALIGN), (dict(k=A + 8), B.NVFP4_ERR_ALIGN), (dict(v=A + 4), B.NVFP4_ERR_ALIGN),
    (dict(q=A + 8), B.NVFP4_ERR_ALIGN), (dict(q_out=ODD), B.NVFP4_ERR_ALIGN), (dict(positions=ODD), B.NVFP4_ERR_ALIGN),
    (dict(freqs=A + 4), B.NVFP4_ERR_ALIGN), (dict(q_out=A, ldqo=4096), B.NVFP4_ERR_ARG), (dict(q_out=A, dtype=0), B.NVFP4_ERR_ARG),
    (dict(tokens=0, k=None, slots=None), B.NVFP4_OK)])
def test_append_refusals(L, over, status):
    d = desc()
    assert L.nvfp4_kv_append(ctypes.byref(append(d, **over)), None) == status


def test_append_and_read_null_and_pool(L):
    assert L.nvfp4_kv_append(None, None) == B.NVFP4_ERR_NULL
    for over, status in ((dict(pool=None), B.NVFP4_ERR_NULL), (dict(pool=A + 8), B.NVFP4_ERR_ALIGN)):
        d = desc(**over)
        assert L.nvfp4_kv_append(ctypes.byref(append(d)), None) == status
        assert L.nvfp4_kv_append(ctypes.byref(append(d, tokens=0)), None) == B.NVFP4_OK
        assert L.nvfp4_kv_read(ctypes.byref(d), A, 4, A, 1024, A, 1024, 1, None) == status
        assert L.nvfp4_attn_decode(ctypes.byref(attn(d)), None) == status
    d = desc()
    r = lambda **o: L.nvfp4_kv_read(ctypes.byref(d), *(dict(slots=A, tokens=4, k=A, ldk=1024, v=A, ldv=1024, dtype=1) | o).values(), None)  # noqa: E731
    assert r(tokens=-1) == r(ldk=1000) == r(ldv=1028) == r(tokens=1 << 25) == B.NVFP4_ERR_SHAPE
    assert r(dtype=2) == B.NVFP4_ERR_DTYPE
    assert r(slots=None) == B.NVFP4_ERR_NULL
    assert r(slots=A + 4) == r(k=A + 8) == r(v=A + 8) == B.NVFP4_ERR_ALIGN
    assert r(tokens=0) == r(k=None, v=None) == B.NVFP4_OK
    assert L.nvfp4_kv_read(None, A, 4, A, 1024, A, 1024, 1, None) == B.NVFP4_ERR_NULL


def attn(d, **over):
    a = B.AttnArgs(cache=ctypes.pointer(d), batch=4, q_heads=40, q=A, ldq=5120, page_table=A, table_width=4, seq_lens=A,
                   scale=0.1, out=2 * A, ldo=5120, workspace=A, workspace_bytes=1 << 40)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), B.NVFP4_ERR_SHAPE), (dict(batch=65537), B.NVFP4_ERR_SHAPE), (dict(q_heads=0), B.NVFP4_ERR_SHAPE),
    (dict(q_heads=12), B.NVFP4_ERR_SHAPE), (dict(q_heads=32776), B.NVFP4_ERR_SHAPE), (dict(table_width=-1), B.NVFP4_ERR_SHAPE),
    (dict(table_width=(1 << 24) + 1), B.NVFP4_ERR_SHAPE), (dict(batch=65536, table_width=1 << 22), B.NVFP4_ERR_SHAPE),
    (dict(batch=65536, q_heads=32768, ldq=1 << 23, ldo=1 << 23, table_width=8), B.NVFP4_ERR_SHAPE),
    (dict(window=-1), B.NVFP4_ERR_ARG), (dict(scale=0.0), B.NVFP4_ERR_ARG),
    (dict(scale=-1.0), B.NVFP4_ERR_ARG), (dict(scale=float("nan")), B.NVFP4_ERR_ARG), (dict(scale=float("inf")), B.NVFP4_ERR_ARG),
    (dict(ldq=5112), B.NVFP4_ERR_SHAPE), (dict(ldo=5124), B.NVFP4_ERR_SHAPE), (dict(q=None), B.NVFP4_ERR_NULL),
    (dict(out=None), B.NVFP4_ERR_NULL), (dict(seq_lens=None), B.NVFP4_ERR_NULL), (dict(page_table=None), B.NVFP4_ERR_NULL),
    (dict(q=A + 8), B.NVFP4_ERR_ALIGN), (dict(out=ODD), B.NVFP4_ERR_ALIGN), (dict(page_table=ODD), B.NVFP4_ERR_ALIGN),
    (dict(seq_lens=ODD), B.NVFP4_ERR_ALIGN), (dict(lse=ODD), B.NVFP4_ERR_ALIGN), (dict(workspace=None), B.NVFP4_ERR_WORKSPACE),
    (dict(workspace_bytes=1024), B.NVFP4_ERR_WORKSPACE), (dict(workspace=A + 8), B.NVFP4_ERR_ALIGN),
    (dict(batch=0, q=None, out=None, workspace=None), B.NVFP4_OK)])
def test_attention_refusals(L, over, status):
    d = desc()
    assert L.nvfp4_attn_decode(ctypes.byref(attn(d, **over)), None) == status


def test_attention_workspace(L):
    n, d = ctypes.c_size_t(), desc()
    assert L.nvfp4_attn_decode_workspace_bytes(ctypes.byref(attn(d)), None) == B.NVFP4_ERR_NULL
    assert L.nvfp4_attn_decode_workspace_bytes(None, ctypes.byref(n)) == B.NVFP4_ERR_NULL
    assert L.nvfp4_attn_decode(None, None) == B.NVFP4_ERR_NULL
    assert L.nvfp4_attn_decode(ctypes.byref(B.AttnArgs()), None) == B.NVFP4_ERR_NULL
    blank = dict(q=None, out=None, page_table=None, seq_lens=None, workspace=None, scale=0.0, ldq=0, ldo=0)
    assert L.nvfp4_attn_decode_workspace_bytes(ctypes.byref(attn(d, **blank)), ctypes.byref(n)) == 0
    need = n.value
    assert need > 1024
    a = attn(d, workspace_bytes=need - 1)
    assert L.nvfp4_attn_decode(ctypes.byref(a), None) == B.NVFP4_ERR_WORKSPACE
    assert str(need).encode() in L.nvfp4_last_error()
    assert L.nvfp4_attn_decode_workspace_bytes(ctypes.byref(attn(d, batch=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert L.nvfp4_attn_decode_workspace_bytes(ctypes.byref(attn(d, table_width=0)), ctypes.byref(n)) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, pos, table = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32), B.RopeTable(torch.zeros(32, dtype=torch.int64), 64, 0, 1.0)
    with pytest.raises(ValueError, match="GPU"):
        B.rope(x, pos, table)
    with pytest.raises(ValueError):
        B.rope(x[0], pos, table)
    with pytest.raises(TypeError):
        B.rope(x.half(), pos, table)
    with pytest.raises(ValueError, match="contiguous"):
        B.rope(torch.zeros(2, 64, 3).transpose(1, 2), pos, table)
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device="cpu")
    k = torch.zeros(2, 1, 64)
    with pytest.raises(ValueError, match="GPU"):
        B.kv_append(cache, k, k, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="heads"):
        B.kv_append(cache, torch.zeros(2, 2, 64), k, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        B.kv_append(cache, k, k.bfloat16(), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        B.kv_read(cache, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        B.attn_decode(k, cache, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


# ---- the tests' own reference ---------------------------------------------------

def test_reference_pins():
    e4m3 = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.E4M3, e4m3)
    x = torch.linspace(0, 500, 100001, dtype=torch.float32)
    assert np.array_equal(R.E4M3[R.nearest(x.clamp(max=448).numpy(), R.E4M3)], x.clamp(max=448).to(torch.float8_e4m3fn).double().numpy())
    assert R.E2M1[R.nearest([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 9], R.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    # Values on the format's grid are stored as they are.
    g = np.random.default_rng(0)
    block = np.append(g.choice(R.E2M1, 15), 6.0)[None].astype(np.float32) * np.float32(0.75)
    assert np.array_equal(R.stored(block, 2), block)
    row = (np.append(g.choice(R.E4M3[64:], 15), 448.0) * 2.0 ** -20)[None].astype(np.float32)
    assert np.array_equal(R.stored(row, 1), row)
    o, lse, _, _ = R.attend(np.zeros((1, 4)), np.ones((8, 4)), np.arange(32.0).reshape(8, 4), 1.0)
    assert np.allclose(o, np.arange(32.0).reshape(8, 4).mean(0)) and np.isclose(lse, math.log(8))
