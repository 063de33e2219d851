"""Calls of the attention side that need no pool, under the sanitizers' build of its host code on the CPU."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CSRC, ENV, HERE, HIPCC, ROOT, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")
def test_calls_without_a_pool(tmp_path):
    import torch
    if torch.cuda.device_count() != 0:
        pytest.skip("a GPU is visible: the library's host code is built and run for a machine without one")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include")]
    srcs = [os.path.join(CSRC, f) for f in ("attn_decode.hip", "kv_cache.hip", "rope.hip", "attn_abi.cpp")]
    srcs.append(os.path.join(HERE, "attn_null_pool_driver.cpp"))

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        run([HIPCC, *flags, "-c", src, "-o", obj])
        return obj
    with ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = str(tmp_path / "attn_null_pool_driver")
    run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
         *objs, "-o", exe])
    r = run([exe], env=ENV)
    assert r.stdout.strip().endswith("ok"), r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
