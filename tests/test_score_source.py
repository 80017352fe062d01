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


def test_barriers_are_set_up_before_anything_meets_them():
    """From a kernel's first mbar_init to the CTA's barrier: both fences, and no copy, product or wait."""
    for name, kernels in (("score_fwd_tc.cu", 1), ("score_bwd_tc.cu", 2)):
        text = open(os.path.join(CSRC, name)).read()
        starts = [m.start() for m in re.finditer(r"for \(int i = 0; i < L::kNumBars; \+\+i\)", text)]
        assert len(starts) == kernels
        for at in starts:
            part = text[at:text.index("__syncthreads();", at)]
            assert part.index("mbar_init(") < part.index("fence_mbar_init();") < part.index("fence_async();"), name
            assert not re.search(r"tma_load|bulk_g2s|expect_tx|mma_|mbar_wait|cluster_peer|next_block", part), name
            # and none earlier in the same function
            head = text[text.rindex("\ntemplate <int D", 0, at):at]
            assert not re.search(r"tma_load\w*\(|bulk_g2s\(|expect_tx\(|mma_\w+\(|mbar_wait\w*\(|cluster_peer\(", head), name
