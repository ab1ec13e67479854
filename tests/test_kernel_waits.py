"""What the kernels' sources must keep in order (read as text: the wrong order
could stop a GPU, so it is never run)."""
import os
import re

import paged_kv_cache_241_gb300 as pkv

CSRC = os.path.join(os.path.dirname(pkv.__file__), "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_prompt_weights_take_tensor_memory_after_the_wait_for_the_kernel_before():
    """The first pass is a programmatic dependent of whatever precedes the call.  Were
    it to take all of tensor memory before it waits, a kernel before it that has yet to
    allocate its own on the same SM would wait for it, and it for that kernel's end."""
    kernel = code("prefill_weights.cu").split("prompt_weights_kernel(", 1)[1]
    first_wait, alloc = kernel.index("griddepcontrol.wait"), kernel.index("tmem_alloc(")
    assert first_wait < alloc
    # unconditionally for all of the first pass's threads
    assert 'if (PASS == 1) asm volatile("griddepcontrol.wait;"' in kernel[:alloc]


def test_the_plan_beside_the_rows_reads_past_the_l1():
    """plan_step's second launch has no wait of its own before it reads lengths, tables and stack, which the step before
    wrote from other SMs: all of its reads go through one function, whose loads leave the SM's L1 out in that launch."""
    text = code("plan_step.cu")
    assert "return kPart == kState ? __ldcg(x) : *x;" in text
    body = text.split("PlanSeq plan_seq(", 1)[1].split('extern "C"', 1)[0]
    arrays = r"p\.(?:new_lens|context_lens|borrowed|block_tables|free_blocks|num_free)\b"
    assert not re.search(r"\*\s*" + arrays, body)
    for m in re.finditer(arrays + r"\[", body):  # (only stores are left)
        depth, at = 1, m.end()
        while depth:
            depth += {"[": 1, "]": -1}.get(body[at], 0)
            at += 1
        assert re.match(r"\s*=[^=]", body[at:]), body[m.start():at]
