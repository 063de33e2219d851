"""GPU parity: the paged key-value cache, written and read back, against the formats' rules."""
import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu

FORMATS = [B.NVFP4_KV_BF16, B.NVFP4_KV_E4M3, B.NVFP4_KV_NVFP4]
IDS = ["bf16", "e4m3", "nvfp4"]


def wide(rng, *shape):
    """N(0, 1) spread over 2^-12 .. 2^12 per head, with zeros of both signs and whole zero rows."""
    x = rng.standard_normal(shape) * np.exp2(rng.uniform(-12, 12, size=shape[:-1] + (1,)))
    x[rng.random(shape) < 0.02] = 0.0
    x[rng.random(shape) < 0.02] = -0.0
    x[rng.random(shape[:-1]) < 0.05] = 0.0
    return x.astype(np.float32)


def rows(x, dtype, dev, pad=24):
    """x [tokens][heads][d] on the device inside wider rows; and its values as float32."""
    t, h, d = x.shape
    buf = torch.full((t, h * d + pad), 7.0, dtype=dtype, device=dev)
    view = buf[:, :h * d].unflatten(1, (h, d))
    view.copy_(torch.from_numpy(x))
    return view, view.float().cpu().numpy()


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 128, 160, 192, 240, 256])
def test_round_trip(fmt, d):
    dev = device()
    rng = np.random.default_rng(d)
    for dtype, tokens, heads, page in ((torch.bfloat16, 37, 3, 16), (torch.float32, 70, 1, 48)):
        pages = tokens // page + 4
        scales = (1.0, 1.0) if fmt != B.NVFP4_KV_NVFP4 else (0.37, 2.5)
        cache = B.KvCache(pages, page, heads, d, fmt, *scales, device=dev)
        cache.pool.fill_(0xff)                                    # the pool needs no initial contents
        k, kh = rows(wide(rng, tokens, heads, d), dtype, dev)
        v, vh = rows(wide(rng, tokens, heads, d), dtype, dev)
        slots = torch.from_numpy(rng.permutation(pages * page)[:tokens]).to(dev)
        B.kv_append(cache, k, v, slots)
        for out in (torch.float32, torch.bfloat16):
            k2, v2 = B.kv_read(cache, slots, dtype=out)
            for got, x, st in ((k2, kh, scales[0]), (v2, vh, scales[1])):
                # The value is one fp32 product (of the code and block scale, exact, with the tensor scale).
                want = torch.from_numpy(R.stored(x, fmt, st)).float().to(out)
                same = got.cpu().eq(want)
                assert same.all(), (dtype, out, np.argwhere(~same.numpy())[:4])


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_every_bf16_magnitude(fmt):
    """Every finite bf16 value beside a row (or block) maximum of several sizes: all codes, borders and ties."""
    dev = device()
    bits = np.arange(0, 0x7f80, dtype=np.uint16)
    vals = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).float().numpy()
    vals = vals[: len(vals) // 15 * 15].reshape(-1, 15)
    for top in (1.0, 6.0, 448.0, 1.75 * 2.0 ** 20, 2.0 ** -9, 3.0e38):
        x = np.concatenate([np.full((len(vals), 1), top, np.float32), np.where(vals <= top, vals, -np.fmod(vals, np.float32(top)))], 1)
        x = x[:, None, :].astype(np.float32)
        cache = B.KvCache(len(x) // 16 + 1, 16, 1, 16, fmt, device=dev)
        t = torch.from_numpy(x).to(dev)
        slots = torch.arange(len(x), device=dev)
        B.kv_append(cache, t, t, slots)
        k, v = B.kv_read(cache, slots, dtype=torch.float32)
        want = torch.from_numpy(R.stored(x, fmt)).float()
        assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want), top


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_not_finite(fmt):
    dev = device()
    x = np.ones((4, 2, 32), np.float32)
    x[1, 0, 3], x[2, 1, 20], x[3, 1, 0] = np.nan, np.inf, -np.inf
    cache = B.KvCache(1, 16, 2, 32, fmt, device=dev)
    t = torch.from_numpy(x).to(dev)
    slots = torch.arange(4, device=dev)
    B.kv_append(cache, t, t, slots)
    for got in B.kv_read(cache, slots, dtype=torch.float32):
        want = torch.from_numpy(R.stored(x, fmt)).float()
        assert torch.equal(got.cpu().nan_to_num(77.0, 78.0, 79.0), want.nan_to_num(77.0, 78.0, 79.0))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_skipped_rows_and_neighbours(fmt):
    """Slots outside the pool are skipped by both directions; other slots keep their bytes."""
    dev = device()
    rng = np.random.default_rng(5)
    cache = B.KvCache(3, 32, 2, 64, fmt, device=dev)
    every = torch.arange(96, device=dev)
    old, _ = rows(wide(rng, 96, 2, 64), torch.float32, dev)
    B.kv_append(cache, old, old, every)
    k0, v0 = B.kv_read(cache, every, dtype=torch.float32)
    new, newh = rows(wide(rng, 6, 2, 64), torch.float32, dev)
    slots = torch.tensor([-1, 17, 96, 95, 2 ** 40, -2 ** 62], device=dev)
    table = B.rope_table(64, device=dev)
    q = torch.randn(6, 4, 64, device=dev)
    q_out = torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device=dev)
    B.kv_append(cache, new, new, slots, positions=torch.zeros(6, dtype=torch.int32, device=dev), table=table, q=q, q_out=q_out)
    k1, v1 = B.kv_read(cache, every, dtype=torch.float32)
    want = torch.from_numpy(R.stored(newh, fmt)).float()
    for old_t, new_t in ((k0, k1), (v0, v1)):
        keep = torch.ones(96, dtype=torch.bool)
        keep[[17, 95]] = False
        assert torch.equal(old_t.cpu()[keep], new_t.cpu()[keep])
        assert torch.equal(new_t.cpu()[[17, 95]], want[[1, 3]])
    assert torch.equal(q_out[[1, 3]], q.to(torch.bfloat16)[[1, 3]])     # position 0: no turn
    assert (q_out[[0, 2, 4, 5]] == 3.0).all()
    out = torch.full((6, 2, 64), 5.0, device=dev)
    B.kv_read(cache, slots, k_out=out)
    assert (out[[0, 2, 4, 5]] == 5.0).all() and torch.equal(out[[1, 3]].cpu(), want[[1, 3]])
    twice = torch.tensor([17, 17, 95], device=dev)
    k2, v2 = B.kv_read(cache, twice, dtype=torch.float32)
    assert torch.equal(k2.cpu(), want[[1, 1, 3]]) and torch.equal(v2, k2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (80, 80), (192, 48), (256, 240)])
def test_rotary_append(layout, d, rot):
    """Keys turned on the way in, queries into q_out, from one fused QKV row; values as they are."""
    dev = device()
    tokens, hq, hk, page = 45, 5, 2, 16
    table = B.rope_table(rot, base=1e6, layout=layout, device=dev)
    g = torch.Generator().manual_seed(d)
    pos = np.arange(900_000, 900_000 + tokens).astype(np.int32)
    for dtype in (torch.bfloat16, torch.float32):
        qkv = torch.randn(tokens, (hq + 2 * hk) * d, generator=g).to(dtype)
        heads = qkv.unflatten(1, (hq + 2 * hk, d))
        dq, dk, dv = heads.to(dev).split([hq, hk, hk], 1)
        x64 = heads.double().numpy()
        turned, size = R.rope(x64[:, :hq + hk], pos, table.freqs.cpu().numpy(), layout == "interleaved")
        p = torch.from_numpy(pos).to(dev)
        slots = torch.from_numpy(np.random.default_rng(1).permutation(80)[:tokens]).to(dev)
        for fmt in FORMATS:
            cache = B.KvCache(5, page, hk, d, fmt, device=dev)
            q_out = B.kv_append(cache, dk, dv, slots, positions=p, table=table, q=dq)
            k, v = (t.double().cpu().numpy() for t in B.kv_read(cache, slots, dtype=torch.float32))
            err = np.abs(q_out.double().cpu().numpy() - turned[:, :hq])
            assert (err <= R.ROPE_STEPS * size[:, :hq] + 2.0 ** -8 * np.abs(turned[:, :hq])).all()
            assert np.array_equal(v, R.stored(heads[:, hq + hk:].float().numpy(), fmt).astype(np.float32))
            want, step = turned[:, hq:], R.ROPE_STEPS * size[:, hq:]
            step[..., rot:] = 0.0       # these only move: exact (and often on a border, as bf16 values are)
            if fmt == B.NVFP4_KV_BF16:
                bound = 2.0 ** -8 * np.abs(want) + step
            else:
                # The fp32 values before the rule are within `step`; where the rule gives the same codes and scales for
                # values that far to either side, the code is settled; the rest may be one grid step off.
                lo, hi = R.stored((want - 4 * step).astype(np.float32), fmt), R.stored((want + 4 * step).astype(np.float32), fmt)
                mid = R.stored(want.astype(np.float32), fmt)
                unsettled = (lo != mid) | (hi != mid)
                assert unsettled.mean() < 0.01
                block = np.abs(want).reshape(*want.shape[:2], -1, 16).max(-1).repeat(16, -1)
                coarse = 2.0 ** -3 * np.abs(want) + block * 2.0 ** -9 if fmt == B.NVFP4_KV_E4M3 else block * (1 / 3 + 2.0 ** -3)
                bound = np.where(unsettled, coarse, 0.0)
                want = mid
            err = np.abs(k - want)
            assert (err <= bound).all(), (dtype, fmt, np.argwhere(err > bound)[:4], (err - bound).max())


def test_queries_in_place_and_empty():
    dev = device()
    table = B.rope_table(64, device=dev)
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_E4M3, device=dev)
    q = torch.randn(3, 4, 64, device=dev).to(torch.bfloat16)
    kv = torch.randn(3, 1, 64, device=dev).to(torch.bfloat16)
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device=dev)
    want = B.rope(q, pos, table)
    got = B.kv_append(cache, kv, kv, torch.arange(3, device=dev), positions=pos, table=table, q=q, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    none = torch.empty(0, 1, 64, device=dev)
    assert B.kv_append(cache, none, none, torch.empty(0, dtype=torch.int64, device=dev)) is None
    k, v = B.kv_read(cache, torch.empty(0, dtype=torch.int64, device=dev))
    assert k.shape == v.shape == (0, 1, 64)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_capture_and_replay(fmt):
    """Writing with rotary positions, reading back and turning, captured together and replayed among eager calls over
    changing rows, positions and slots."""
    dev = device()
    g = torch.Generator().manual_seed(fmt)
    tokens, hq, hk, d = 37, 5, 2, 128
    table = B.rope_table(d, device=dev)
    caches = [B.KvCache(6, 16, hk, d, fmt, device=dev) for _ in range(2)]
    for c in caches:
        c.pool.zero_()
    qkv = torch.empty(tokens, hq + 2 * hk, d, dtype=torch.bfloat16, device=dev)
    pos = torch.empty(tokens, dtype=torch.int32, device=dev)
    slots = torch.empty(tokens, dtype=torch.int64, device=dev)

    def step(cache):
        q, k, v = qkv.split([hq, hk, hk], 1)
        q_out = B.kv_append(cache, k, v, slots, positions=pos, table=table, q=q)
        return q_out, *B.kv_read(cache, slots), B.rope(qkv, pos, table, inverse=True)

    def new_inputs():
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        pos.copy_(torch.randint(0, 2 ** 31 - 1, (tokens,), generator=g))
        slots.copy_(torch.randperm(96, generator=g)[:tokens])

    new_inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(caches[0])
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            captured = step(caches[0])
    torch.cuda.synchronize()
    for _ in range(4):
        new_inputs()
        graph.replay()
        eager = step(caches[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
