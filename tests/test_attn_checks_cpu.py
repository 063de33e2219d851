"""The attention side's argument checks without a GPU, beyond those of test_attn_abi_cpu.py."""
import ctypes

import pytest
import torch

from bit_quantized_decode_amd import binding as B
from test_attn_abi_cpu import L, attn, desc  # noqa: F401


@pytest.mark.parametrize("scale,status", [(2.0 ** 127, B.NVFP4_ERR_WORKSPACE), (1.001 * 2.0 ** 127, B.NVFP4_ERR_ARG),
                                          (3.4e38, B.NVFP4_ERR_ARG), (1e-45, B.NVFP4_ERR_WORKSPACE)])
def test_softmax_scale(L, scale, status):  # noqa: F811
    """Up to 2^127, with which the product with log2 e is still a number (a call without a workspace stops there)."""
    d = desc()
    assert L.nvfp4_attn_decode(ctypes.byref(attn(d, scale=scale, workspace=None)), None) == status


@pytest.mark.parametrize("freqs,error", [
    (torch.zeros(31, dtype=torch.int64), ValueError), (torch.zeros(1, dtype=torch.int64).expand(32), ValueError),
    (torch.zeros(64, dtype=torch.int64)[::2], ValueError), (torch.zeros(0, dtype=torch.int64), ValueError),
    (torch.zeros(32, dtype=torch.float64), TypeError), (torch.zeros(64, dtype=torch.int32), TypeError),
    (torch.zeros(32, dtype=torch.int64), None), (torch.zeros(40, dtype=torch.int64), None),
    (torch.zeros(4, 8, dtype=torch.int64), None), (torch.zeros(32, dtype=torch.int64).view(torch.uint64), None)])
def test_a_table_of_the_callers_own(freqs, error):
    """A table that does not hold rot_dim / 2 frequencies is refused (a right one is refused for lying on the CPU)."""
    table = B.RopeTable(freqs, 64, B.NVFP4_ROPE_HALF, 1.0)
    x, pos = torch.zeros(2, 1, 64), torch.zeros(2, dtype=torch.int32)
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device="cpu")
    for call in (lambda: B.rope(x, pos, table),
                 lambda: B.kv_append(cache, x, x, torch.zeros(2, dtype=torch.int64), positions=pos, table=table)):
        with pytest.raises(error or ValueError, match="rotary table" if error else "GPU"):
            call()


@pytest.mark.parametrize("prepared", [False, True])
def test_a_workspace_that_is_not_contiguous(prepared):
    """An expanded workspace has less memory than elements: refused (a contiguous one is refused for lying on the CPU)."""
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device="cpu")
    q, table, lens = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    call = B.attn_decode_prepared if prepared else B.attn_decode
    for ws, match in ((torch.zeros(1, dtype=torch.uint8).expand(1 << 24), "contiguous"),
                      (torch.zeros(1 << 10, 4, dtype=torch.uint8)[:, :2], "contiguous"), (torch.zeros(1 << 10), "GPU")):
        with pytest.raises(ValueError, match=match):
            call(q, cache, table, lens, ws=ws)


def test_rope_out_of_another_dtype():
    """Given both, out and dtype have to agree (and if they do, the call is refused for lying on the CPU)."""
    table = B.RopeTable(torch.zeros(32, dtype=torch.int64), 64, B.NVFP4_ROPE_HALF, 1.0)
    x, pos, out = torch.zeros(2, 1, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    for call in (B.rope, B.rope_prepared):
        with pytest.raises(TypeError, match="dtype"):
            call(x, pos, table, out=out, dtype=torch.float32)
        for dtype in (None, torch.bfloat16):
            with pytest.raises(ValueError, match="GPU"):
                call(x, pos, table, out=out, dtype=dtype)


@pytest.mark.parametrize("lse", [1, "yes", [True]])
def test_lse_of_another_kind(lse):
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device="cpu")
    q, table, lens = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (B.attn_decode, B.attn_decode_prepared):
        with pytest.raises(TypeError, match="lse"):
            call(q, cache, table, lens, lse=lse)


@pytest.mark.parametrize("rot,base,trained,fast,slow", [(64, 1e4, 4, 32.0, 1.0), (16, 1e6, 6.28, 2.0, 1.0), (128, 1e4, 100, 1e3, 40.0),
                                                        (32, 1e4, 1e-3, 32.0, 1.0)])
def test_yarn_with_every_pair_slow(L, rot, base, trained, fast, slow):  # noqa: F811
    """Trained over so few positions that even the first pair turns less than beta_slow times: all pairs are f / factor."""
    assert trained / (2 * 3.141592653589793) < slow
    got, magnitude = B.rope_freqs(rot, base, ("yarn", 8.0, trained, fast, slow))
    want, _ = B.rope_freqs(rot, base, ("linear", 8.0))
    # Two roundings of the table's last bit, and of its extended-precision operations.
    assert ((got - want).abs().double() <= 1 + want.double() * 2.0 ** -58).all()
    assert magnitude == pytest.approx(0.1 * 2.0794415416798357 + 1.0, rel=2.0 ** -24)
