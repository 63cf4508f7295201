"""Launches chained by programmatic launch: griddepcontrol.wait is what makes an earlier launch's
results visible, so every kernel of the cache attention waits before it reads any of them."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "random_feature_linear_b200", "csrc")
# what reads the workspace: queries, list of ranges, partial results
READS = r"\bitem_of\(|\bat<|\bsched_\w+\(|\bvisible_keys\("


def kernels():
    """(file, name, body) of the cache attention's kernels."""
    for f in ("cache_attend.cu", "cache_attend_mma.cu", "cache_attend_tc.cu", "cache_queries.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        for m in re.finditer(r"__global__.*?(\w+_kernel)\(", text, re.S):
            depth, i = 0, text.index("{", m.end())
            begin = i
            while True:
                depth += (text[i] == "{") - (text[i] == "}")
                i += 1
                if depth == 0:
                    break
            yield f, m.group(1), text[begin:i]


def test_kernels_wait_before_they_read_the_workspace():
    seen = set()
    for f, name, body in kernels():
        seen.add(name)
        if name in ("queries_kernel", "queries_mma_kernel"):       # the first launch
            continue
        wait = re.search(r"^  pdl_wait\(\);", body, re.M)          # (unconditional)
        assert wait, (f, name)
        before = body[:wait.start()]
        if name == "range_tc_kernel":
            # an item of the prefix alone is made of the call's parameters
            before = before.replace("item_of(q, blockIdx.x, hk, RT * kT, true, false)", "")
        assert not re.search(READS, before), (f, name)
    assert seen == {"queries_kernel", "queries_mma_kernel", "range_kernel", "range_mma_kernel",
                    "range_tc_kernel", "join_kernel"}
