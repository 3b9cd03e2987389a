"""Orders in the kernel sources that no run can show safely: what would go wrong is a GPU that hangs."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_gqa_min_b200", "csrc")


def code(name: str) -> str:
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_the_next_kernel_starts_after_tensor_memory_is_held():
    """A CTA that lets the next kernel start before it holds its tensor memory can lose it to that kernel's
    CTA on the same SM, which keeps it while it waits for this one.  One thread's launch_dependents counts for
    its CTA, so a barrier has to lie between the allocation and any thread's trigger."""
    seen = 0
    for part in code("weights.cu").split("__global__")[1:]:
        if "tc::alloc(" not in part:
            continue
        seen += 1
        between = part[part.index("tc::alloc("):part.index("pdl_trigger()")]
        assert part.index("pdl_trigger()") > part.index("tc::alloc(")
        assert "__syncthreads()" in between
    assert seen == 1


def test_waits_before_full_warp_operations_have_one_verdict():
    """The four-bit attention and the tensor-memory weights go on with full-mask shuffles and warp-wide MMAs
    after a wait, so all lanes have to give up together or not at all."""
    for name in ("kv4_decode.cu", "weights.cu"):
        text = code(name)
        assert re.findall(r"\bmbar_wait_warp\(", text), name
        assert not re.findall(r"\bmbar_wait\(|\bmbar_wait_sleep\(", text), name


def test_bad_arguments_of_the_warp_wait_test():
    from block_sparse_gqa_min_b200 import sba

    call = sba.load().sba_selftest_wait_vote
    for status, verdicts, limit in ((None, 0x1000, 1000), (0x1000, None, 1000), (0x1000, 0x2000, 0),
                                    (0x1000, 0x2000, 1_000_000_001)):
        assert call(status, verdicts, limit, None) == sba.SBA_ERR_INVALID_ARG


def test_a_weights_call_that_says_ok_has_launched():
    """Whatever the thresholds between the two kernels are: no way through the dispatch returns SBA_OK by
    itself, and a call with a gate bias never goes to the kernel that takes none."""
    text = code("weights.cu")
    dispatch = text[text.index("int launch_weights("):]
    dispatch = dispatch[:dispatch.index("\n}\n")]
    assert "return SBA_OK" not in dispatch
    conditions = re.findall(r"if \(([^{]*a\.rows >= least)\) \{", dispatch)
    assert conditions == ["!gate_bias && a.rows >= least"]
    assert "gate_bias" not in text[text.index("void __launch_bounds__(kTcThreads, 2)"):text.index("int launch_weights(")]
