"""AddressSanitizer / UndefinedBehaviorSanitizer build of the host code of nvfp4_attn_long.h's entry points, on the CPU:
arguments that they must refuse before any launch, and the size queries."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CSRC, ENV, HERE, HIPCC, ROOT, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")
def test_long_cache_abi_host_code_under_asan_and_ubsan(tmp_path):
    import torch
    if torch.cuda.device_count() != 0:
        pytest.skip("a GPU is visible: the driver's placeholder pointers are for a machine without one")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include")]
    srcs = [os.path.join(CSRC, f) for f in ("attn_decode.hip", "attn_shared.hip", "attn_pages.hip", "kv_bounds.hip", "kv_select.hip",
                                            "attn_long_abi.cpp", "kv_cache.hip", "rope.hip", "attn_abi.cpp", "abi.cpp", "pack.hip",
                                            "quantize.hip", "gemv.hip", "skinny.hip", "prefill.hip", "moe.hip", "w4a4.hip")]
    srcs.append(os.path.join(HERE, "attn_long_abi_driver.cpp"))

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        run([HIPCC, *flags, "-c", src, "-o", obj])
        return obj
    with ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = str(tmp_path / "attn_long_abi_driver")
    run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
         *objs, "-o", exe])
    r = run([exe], env=ENV)
    assert r.stdout.strip().endswith("ok"), r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
