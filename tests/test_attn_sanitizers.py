"""AddressSanitizer / UndefinedBehaviorSanitizer build of the attention side's
host code on the CPU: every entry point with arguments it must refuse before
any launch, and the host-only calls.  The HIP sources are compiled in full, with
the sanitizers on their host side only (-Xarch_host)."""
import os

import pytest

from test_sanitizers import CSRC, ENV, HERE, HIPCC, ROOT, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")
def test_attention_abi_host_code_under_asan_and_ubsan(tmp_path):
    import torch
    if torch.cuda.device_count() != 0:
        pytest.skip("a GPU is visible: the driver's placeholder pointers are for a machine without one")
    from concurrent.futures import ThreadPoolExecutor
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include")]
    srcs = [os.path.join(CSRC, f) for f in ("rope.hip", "kv_cache.hip", "attn_decode.hip", "attn_abi.cpp", "abi.cpp",
                                            "pack.hip", "quantize.hip", "gemv.hip", "skinny.hip", "prefill.hip", "moe.hip",
                                            "w4a4.hip")]
    srcs.append(os.path.join(HERE, "attn_abi_driver.cpp"))

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        run([HIPCC, *flags, "-c", src, "-o", obj])
        return obj
    with ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, srcs))
    exe = str(tmp_path / "attn_abi_driver")
    run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
         *objs, "-o", exe])
    r = run([exe], env=ENV)
    assert r.stdout.strip().endswith("ok"), r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
