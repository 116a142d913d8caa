"""Hand-over of operand tiles between the two CTAs of a pair, read from the kernels' source: a relaxed remote
arrive orders no ordinary store, so tiles that warps store themselves reach the other CTA's tensor-core issue
only through a fence at cluster scope, by a thread that has acquired the storing warps' local phases.  (On a
GPU a missing one shows as rare wrong sums, if at all.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_kv_top_gb300", "csrc")


def body(name, start):
    """The brace block that opens first at or after `start` in a source file, without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    at = src.index(start)
    i = src.index("{", at)
    depth = 0
    for j in range(i, len(src)):
        depth += {"{": 1, "}": -1}.get(src[j], 0)
        if depth == 0:
            return src[at:j + 1]
    raise AssertionError(f"{start}: unbalanced")


def test_warps_that_store_tiles_arrive_on_their_own_cta():
    producers = body("tree_common.cuh", "__device__ __forceinline__ void produce_tiles")
    assert "st.shared" in producers and "fence_proxy_async_smem" in producers
    assert "cluster" not in producers.replace("cluster_wait_all", "")
    kernel = body("tree.cu", "tree_dense_kernel")
    for bar in ("q_full", "k_full", "v_full"):  # remote arrives on these only where a fence comes first
        for m in re.finditer(r"mbar_arrive_cluster\(pair_addr\(&(bars\.)?(full|%s)\b" % bar, kernel):
            lead = kernel[:m.start()]
            assert "fence_cluster()" in lead or "auto forward" in lead[-200:], kernel[m.start() - 200:m.end()]


def test_the_fence_is_at_cluster_scope_and_the_issuer_acquires_there():
    assert "fence.acq_rel.cluster" in body("ptx.cuh", "void fence_cluster")
    kernel = body("tree.cu", "tree_dense_kernel")
    issue = kernel[kernel.index("auto issue_qk"):kernel.index("auto stored")]
    waits = re.findall(r"mbar_wait_poll(<\w+>)?\(&bars\.(q|k|v)_full", issue)
    assert len(waits) == 3 and not any(scope for scope, _ in waits)  # the default acquires at cluster scope
    forward = kernel[kernel.index("auto stored"):]
    loop = forward[forward.index("for (int j = -1"):forward.index("__syncwarp")]
    assert loop.index("stored(") < loop.index("fence_cluster()") < loop.index("mbar_arrive_cluster") < loop.index("forward(bars")
