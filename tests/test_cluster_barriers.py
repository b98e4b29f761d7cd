"""The aligned barriers of the page kernels' cluster: an aligned barrier is one
instruction of a whole warp, and lanes that left a loop at different times need
not be together when they come to it.  Read from the source, as nothing on a GPU
is to run without it."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_warps_are_brought_together_before_aligned_cluster_barriers():
    text = open(os.path.join(ROOT, "diffusion_transformer_mlp_gb300", "csrc", "mx_pages.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    barriers = [m.start() for m in re.finditer(r"asm volatile\(\"barrier\.cluster\.\w+\.\w+\.aligned", text)]
    assert len(barriers) >= 2
    for at in barriers:
        before = text[:at].rstrip()
        assert before.endswith("__syncwarp();"), text[max(0, at - 120):at + 60]
