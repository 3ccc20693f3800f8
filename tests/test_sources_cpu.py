"""What the kernels' sources have to keep, read from them (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_lm_head_linear_gb300", "csrc")


def test_warp_aligned_instructions_are_issued_by_a_whole_warp():
    """An instruction with .aligned is undefined, and a barrier among them may never end, where a warp's lanes are
    apart: after a branch that differs by lane nothing but __syncwarp brings them together for certain. So each such
    instruction stands in a function of its own that begins with it."""
    src = open(os.path.join(CSRC, "sm100_ptx.cuh")).read()
    bodies = re.findall(r"__device__ __forceinline__ \w+ (\w+)\([^{]*\) \{\n(.*?)\n\}", src, flags=re.S)
    aligned = {name: body for name, body in bodies if re.search(r'"[^"]*\.aligned', body)}
    assert {"cluster_sync_all", "tmem_ld_wait", "tmem_alloc_pair"} <= set(aligned)
    assert sum(len(re.findall(r'"[^"]*\.aligned', b)) for b in aligned.values()) == len(re.findall(r'"[^"]*\.aligned', src))
    for name, body in aligned.items():
        assert body.lstrip().startswith("__syncwarp();"), name
    for file in os.listdir(CSRC):
        if file != "sm100_ptx.cuh" and file.endswith((".cu", ".cuh", ".h")):
            assert not re.search(r'"[^"]*\.aligned', open(os.path.join(CSRC, file)).read()), file
