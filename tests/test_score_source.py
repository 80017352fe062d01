"""Orders that a GPU run cannot show: an aligned barrier that a warp meets in
parts is undefined, so it may also pass."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_attention_dits_gb300", "csrc")


def functions(name):
    """{function name: body} of the one-purpose device helpers of a file."""
    text = open(os.path.join(CSRC, name)).read()
    found = {}
    for m in re.finditer(r"__device__ __forceinline__ \w+ (\w+)\([^)]*\) \{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        found[m.group(1)] = text[m.end():at]
    return found


def test_warps_converge_before_aligned_barriers():
    for name, fn, what in (("cp_ptx.cuh", "cluster_sync", "barrier.cluster.arrive.release.aligned"),
                           ("score_attn_f32.cu", "group_sync", "bar.sync")):
        body = functions(name)[fn]
        assert what in body and "__syncwarp();" in body and body.index("__syncwarp();") < body.index(what), (name, fn)
