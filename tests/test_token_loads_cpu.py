"""The token-step kernels begin while the kernel in front of them ends, so what they read may still be written then."""
import os
import re

import pytest

from diffusion_transformer_image_mmdit_gb300 import build


@pytest.mark.parametrize("name", ["token_linear.cu", "kv_cache.cu"])
def test_kernels_that_begin_early_use_no_non_coherent_loads(name):
    with open(os.path.join(build.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "launch_after(" in code
    assert not re.search(r"__ldg\b|ld\.global\.nc", code)
    # a kernel that lets the next one start has waited before
    for body in re.findall(r"__global__(.*?)\n}\n", code, re.S):
        if "grid_release()" in body:
            assert body.index("grid_wait()") < body.index("grid_release()")
            assert "__restrict__" not in body
