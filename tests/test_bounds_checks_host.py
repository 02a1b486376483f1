"""Every source file with a count of failed bounds checks makes such checks."""
import os
import re

from paged_kv_cache_xs_gb300 import build as xsbuild


def test_files_with_a_counter_have_checks():
    counted = []
    for name in xsbuild.SOURCES:
        text = open(os.path.join(xsbuild.CSRC, name)).read()
        text = re.sub(r"//[^\n]*", "", text)
        kernels = len(re.findall(r"__global__", text))
        checks = len(re.findall(r"XS_BOUNDS\(", text))
        if "XS_DEFINE_BOUNDS_COUNTER" in text:
            counted.append(name)
            # (slot_mapping_kernel of kv_append.cu writes by its thread's index alone)
            want = 1 if name in ("kv_append.cu", "paged_prefill_tc.cu") else kernels
            assert checks >= want, f"{name}: {checks} checks in {kernels} kernels"
    assert {"qk_norm_rope.cu", "kv4_cache.cu", "kv4_decode.cu", "block_share.cu"} <= set(counted)
