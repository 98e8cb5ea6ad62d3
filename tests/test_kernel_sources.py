"""What the kernel sources may not hold, whatever they compute (no GPU needed)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_step_kv_gb300", "csrc")
SOURCES = sorted(f for pattern in ("*.cu", "*.cuh") for f in glob.glob(os.path.join(CSRC, pattern)))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_into_several_ctas(path):
    """Every rank of a run on several GPUs loads the one library, and a cache pointer does not tell which GPU
    serves its memory: a load into the shared memory of several CTAs at once must not be among its kernels."""
    with open(path) as f:
        text = re.sub(r'"\s*\n\s*"', "", f.read())          # PTX split over adjacent string literals
    found = [m.group(0)[:120] for m in re.finditer(r"cp\.async\.bulk[^\n]*", text) if "multicast" in m.group(0)]
    assert not found


def test_sources_are_there():
    assert {"fa_decode.cu", "fa_prefill.cu", "fa_common.cuh"} <= {os.path.basename(f) for f in SOURCES}
