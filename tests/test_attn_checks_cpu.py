"""The attention side's argument checks without a GPU, beyond those of test_attn_abi_cpu.py."""
import ctypes

import pytest

from bit_quantized_decode_amd import binding as B
from test_attn_abi_cpu import L, attn, desc  # noqa: F401


@pytest.mark.parametrize("scale,status", [(2.0 ** 127, B.NVFP4_ERR_WORKSPACE), (1.001 * 2.0 ** 127, B.NVFP4_ERR_ARG),
                                          (3.4e38, B.NVFP4_ERR_ARG), (1e-45, B.NVFP4_ERR_WORKSPACE)])
def test_softmax_scale(L, scale, status):  # noqa: F811
    """Up to 2^127, with which the product with log2 e is still a number (a call without a workspace stops there)."""
    d = desc()
    assert L.nvfp4_attn_decode(ctypes.byref(attn(d, scale=scale, workspace=None)), None) == status
