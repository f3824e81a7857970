"""Kernels start beside the end of the one before (programmatic launch) and wait for it in the
kernel.  TMEM is taken behind that wait: a kernel before that takes its own late would
otherwise wait for columns that are held until it ends, and neither would."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tmem_is_taken_behind_the_wait_for_the_kernel_before():
    seen = []
    for path in glob.glob(os.path.join(ROOT, "encoder_only_transformer_gb300", "csrc", "*.cu")):
        for body in re.findall(r"__global__.*?\n}\n", open(path).read(), flags=re.S):
            code = re.sub(r"//[^\n]*", "", body)
            if "tmem_alloc" in code:
                assert 0 <= code.find("pdl_wait()") < code.index("tmem_alloc"), path
                seen.append(os.path.basename(path))
    assert {"linear.cu", "linear_rows.cu", "attn_cross.cu", "attn_global.cu", "attn_local.cu"} <= set(seen)
