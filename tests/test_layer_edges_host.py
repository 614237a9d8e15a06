"""Properties of the attention half's sources, refusals and bookkeeping that need no GPU."""
import os
import re

from mtp_speculative_draft_head_gb300 import build


def source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_prompt_kernel_joins_its_warps_by_bounded_waits_only():
    """A warp that gives up leaves its role at once: a barrier of several warps in front of the kernel's last one would hold
    the others for ever. The whole CTA's barrier stands at the start and at the end, outside of every role."""
    text = source("attention_prompt.cu")
    assert "named_barrier" not in text and "bar.sync" not in text and "barrier.sync" not in text
    kernel = text.split("attention_prompt_kernel(const __grid_constant__")[1].split("bool encode_rows")[0]
    roles = kernel.index("if (warp >= 8) {"), kernel.rindex("give_up();")
    at = [i.start() for i in re.finditer(r"__syncthreads\(\)", kernel)]
    assert len(at) == 2 and at[0] < roles[0] and at[1] > roles[1]
    wait = kernel[kernel.index("auto come ="):]  # polls stand in the bounded wait alone
    wait = wait[:wait.index("};")]
    assert kernel.count("mbar_try_wait") == wait.count("mbar_try_wait") and "<= p.wait_ns" in wait


def test_prompt_kernel_lets_an_answer_under_way_land():
    """The answer about the next piece is written into shared memory by the hardware: a wait for it that runs out is
    followed by one with the full limit before the warp leaves."""
    text = source("attention_prompt.cu")
    asked = text.split("clusterlaunchcontrol.try_cancel")[1].split("clusterlaunchcontrol.query_cancel")[0]
    waits = re.findall(r"(come|mbar_wait_bounded)\(smem_addr\(asked\), turn\)", asked)
    assert waits == ["come", "mbar_wait_bounded"]
    assert asked.index("break;") > asked.rindex("mbar_wait_bounded")


def test_scales_that_leave_fp32_with_their_factors_are_refused():
    """scale log2(e) and, over the cache, half of a query row's power of two are fp32 numbers: beyond 2^60 they need not be."""
    import ctypes

    import mtp_speculative_draft_head_gb300 as m
    import test_layer_host as h
    lib = m.load()
    for scale in (2.0 ** 60 * (1 + 2.0 ** -23), 2.0 ** 100, 3.0e38):
        assert ctypes.c_float(scale).value > 2.0 ** 60
        assert h.attend(lib, dict(h.spread(h.ATT), **dict(h.ATT_SIZES, scale=scale))) == m.ERR_ARG
        assert h.prompt(lib, dict(h.spread(h.PROMPT), **dict(h.PROMPT_SIZES, scale=scale))) == m.ERR_ARG
