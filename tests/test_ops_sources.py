"""What the sources of the operators promise by their text."""
import os
import re

from routed_expert_ffn_06_b200 import build


def test_tensor_memory_loads_follow_a_warp_barrier():
    """A wait lets the lanes of a warp go apart; tcgen05.ld is an instruction of
    the whole warp, so the wait for an accumulator ends in a warp barrier."""
    src = open(os.path.join(build.OPS, "fp8_gemm.cu")).read()
    waits = re.findall(r"pipe_wait\(&accf\[[^;]*;\s*([^\n]*)", src)
    assert len(waits) == 2 and all(w.startswith("__syncwarp();") for w in waits)
