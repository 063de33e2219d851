"""The attention side as a decode layer runs it: QKV product, keys and queries turned and the cache written in one call,
attention over the cache, O product -- several steps, against a 64-bit chain over what the cache holds."""
import numpy as np
import pytest
import torch

import attn_reference as R
import oracle
from bit_quantized_decode_amd import binding as B
from bit_quantized_decode_amd import inputs as I
from helpers import TOL, device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [B.NVFP4_KV_BF16, B.NVFP4_KV_E4M3, B.NVFP4_KV_NVFP4], ids=["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("users", [1, 5])
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_decode_steps(fmt, users, graph):
    dev = device()
    hidden, hq, hk, d, page, prompt, steps = 256, 10, 2, 64, 16, 21, 4
    rng = np.random.default_rng(users)
    qkv_n, o_k = (hq + 2 * hk) * d, hq * d
    wqkv, wo = I.nvfp4_matrix(I.GEMV_1K, 7, qkv_n, hidden), I.nvfp4_matrix(I.GEMV_1K, 8, hidden, o_k)
    pqkv, po = (B.pack(torch.from_numpy(c).to(dev), torch.from_numpy(s).to(dev)) for c, s in (wqkv, wo))
    st = I.TENSOR_SCALE
    table = B.rope_table(d, base=1e6, layout="half", device=dev)
    width = -(-(prompt + steps) // page)
    cache = B.KvCache(users * width, page, hk, d, fmt, device=dev)
    cache.pool.fill_(0xff)
    pages = torch.from_numpy(rng.permutation(users * width).reshape(users, width).astype(np.int32)).to(dev)

    def slots_of(user, pos):
        return pages.long()[user, pos // page] * page + pos % page

    def split(rows):
        return rows.unflatten(1, (hq + 2 * hk, d)).split([hq, hk, hk], 1)

    # Prompt: every user's first tokens in one call.
    user, pos = (torch.from_numpy(a.ravel()).to(dev) for a in np.meshgrid(np.arange(users), np.arange(prompt), indexing="ij"))
    x = torch.from_numpy(rng.standard_normal((users * prompt, hidden)).astype(np.float32)).to(torch.bfloat16).to(dev)
    qkv = B.gemm(pqkv, qkv_n, hidden, st, x)
    q, k, v = split(qkv)
    B.kv_append(cache, k, v, slots_of(user, pos), positions=pos.int(), table=table)

    # Decode: fixed buffers, as a captured step has them.
    x = torch.empty(users, hidden, dtype=torch.bfloat16, device=dev)
    lens = torch.full((users,), prompt, dtype=torch.int32, device=dev)
    positions = torch.empty(users, dtype=torch.int32, device=dev)
    slots = torch.empty(users, dtype=torch.int64, device=dev)
    everyone = torch.arange(users, device=dev)
    res = {}

    def step():
        res["qkv"] = B.gemm(pqkv, qkv_n, hidden, st, x, y_dtype=torch.float32)
        q, k, v = split(res["qkv"])
        res["q"] = B.kv_append(cache, k, v, slots, positions=positions, table=table, q=q)
        res["o"] = B.attn_decode(res["q"], cache, pages, lens)
        res["y"] = B.gemm(po, hidden, o_k, st, res["o"].view(users, o_k), y_dtype=torch.float32)

    g = None
    for i in range(steps):
        x.copy_(torch.from_numpy(rng.standard_normal((users, hidden)).astype(np.float32)))
        positions.copy_(lens)
        slots.copy_(slots_of(everyone, lens.long()))
        lens.add_(1)
        if not graph:
            step()
        elif g is None:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            step()                       # writes the same slots as the first replay
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                step()
            g.replay()
        else:
            g.replay()
        torch.cuda.synchronize()

        # The QKV rows, turned, as the cache holds them: each stage against 64 bits from what the stage before wrote.
        y_ref, s = oracle.gemm(wqkv[0], wqkv[1], st, x.cpu().view(torch.int16).numpy().view(np.uint16))
        got = res["qkv"].double().cpu().numpy()
        assert (np.abs(got - y_ref) <= TOL * s).all()
        heads = got.reshape(users, hq + 2 * hk, d)
        turned, size = R.rope(heads[:, :hq + hk], positions.cpu().numpy(), table.freqs.cpu().numpy(), False)
        q64 = res["q"].double().cpu().numpy()
        assert (np.abs(q64 - turned[:, :hq]) <= R.ROPE_STEPS * size[:, :hq] + 2.0 ** -8 * np.abs(turned[:, :hq])).all()
        for u in range(users):
            n = int(lens[u])
            ck, cv = (t.double().cpu().numpy() for t in B.kv_read(cache, slots_of(u, torch.arange(n, device=dev)), dtype=torch.float32))
            assert np.array_equal(cv[n - 1], R.stored(heads[u, hq + hk:].astype(np.float32), fmt).astype(np.float32))
            # The new key: within one step of the format (2^-8, 2^-3 of a value, a third of a block's largest).
            coarse = {0: 2.0 ** -8, 1: 2.0 ** -3, 2: 0.5}[fmt]
            assert (np.abs(ck[n - 1] - turned[u, hq:]) <= coarse * np.abs(turned[u, hq:]).max() + 1e-6).all()
            for h in range(hk):
                rows = slice(h * hq // hk, (h + 1) * hq // hk)
                o, lse, pv, sz = R.attend(q64[u, rows], ck[:, h], cv[:, h], d ** -0.5)
                bound, _ = R.attend_bounds(sz, n, d, o, pv, lse, fmt)
                assert (np.abs(res["o"][u, rows].double().cpu().numpy() - o) <= bound).all(), (i, u, h)
        o_bits = res["o"].reshape(users, o_k).cpu().view(torch.int16).numpy().view(np.uint16)
        y_ref, s = oracle.gemm(wo[0], wo[1], st, o_bits)
        assert (np.abs(res["y"].double().cpu().numpy() - y_ref) <= TOL * s).all()
