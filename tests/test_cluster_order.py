"""Order of the cluster meetings in the chunk kernel, read from its source: CUDA lets a CTA touch another's shared memory
only once that one runs, and a missing wait shows on no device that starts them together."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_block_quantized_moe_b200", "csrc")


def body(text, name):
    """The braces' content of the function `name`, comments removed."""
    text = re.sub(r"//[^\n]*", "", text)
    at = text.index("{", text.index(name + "("))
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
        i += 1


def test_chunk_kernel_waits_for_its_cluster_before_it_writes_there():
    with open(os.path.join(CSRC, "attn_tc.cu")) as f:
        kernel = body(f.read(), "attn_tc_kernel")
    store = kernel.index("cluster_store2(")
    assert kernel.count("cluster_store2(") == 1 and "cluster_store(" not in kernel
    # all threads arrive once, after the only return, and every path waits once before its meeting and the store
    arrive = kernel.index("cluster_started();")
    assert kernel.count("cluster_started();") == 1 and kernel.rindex("return;") < arrive
    waits = [m.start() for m in re.finditer(r"cluster_wait_started\(\);", kernel)]
    meets = [m.start() for m in re.finditer(r"cluster_meet\(\);", kernel)]
    split = kernel.index("setmaxnreg.inc")  # the softmax warps' branch; before it the other warps'
    assert len(waits) == len(meets) == 2
    assert arrive < waits[0] < meets[0] < split < waits[1] < store < meets[1]
    # none of them under a condition that not all threads of the cluster share
    for at in [arrive] + waits + meets:
        head = kernel[:at].rstrip()
        assert head.endswith("if (clustered)") or re.search(r"if \(clustered\) \{[^{}]*$", head), head[-80:]
