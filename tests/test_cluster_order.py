"""Shared memory of another CTA may be touched only once that CTA is known to
run: in the kernels' sources, a barrier of the cluster stands before the first
access to it (a CTA that stored into one that had not begun could lose the
store, or fault; no run shows reliably that it does not)."""
import glob
import os
import re

from paged_kv_cache_177_gb300.build import CSRC


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_where_other_ctas_are_reached():
    """Only these two files do; what follows looks at both."""
    reach = {os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu*")) if "map_shared_rank" in source(f)}
    assert reach == {"pkv_verify.cuh", "pkv_prefill_scored.cuh"}


def test_verification():
    text = source("pkv_verify.cuh")
    kernel = text[text.index("verify_drafts_kernel"):]
    assert kernel.count("map_shared_rank") == 1 and kernel.count("cluster_arrive();") == 1
    # all threads arrive behind the return that a whole cluster takes, and before the walk ...
    left, arrive, begin = kernel.index("return;"), kernel.index("cluster_arrive();"), kernel.index("auto pass = ")
    assert left < arrive < begin and "return" not in kernel[arrive:begin]
    # ... and wait in the first pass, outside the branch that stores
    body = kernel[begin:kernel.index("cluster.sync();", begin)]
    wait, store = body.index("if (passes == 0) cluster_wait();"), body.index("map_shared_rank")
    assert wait < body.index("passes++") < body.index("if (warp == 0") < store
    # no thread leaves before a pass: the walk ends with one
    walk = kernel[kernel.index("cluster.sync();", begin):kernel.index("if (!summed) Z = pass(node, A);")]
    assert walk.count("return") == walk.count("return total;") + walk.count("return __any_sync")


def test_prefill():
    text = source("pkv_prefill_scored.cuh")
    kernel = text[text.index("prefill_scored_kernel("):]
    assert "map_shared_rank" not in kernel
    assert re.search(r"cluster_barrier\(\);\s*scored_join<D>\(", kernel) and kernel.count("scored_join<D>(") == 1
