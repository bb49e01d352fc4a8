"""Bounded waits in the kernels' sources: what a wait that runs out must not leave behind (no GPU needed)."""
import os
import re

import pytest

from video_dit_quantized_b200 import build

KERNELS = {"sparse.cu": 1, "attention.cu": 2, "linear.cu": 2, "select.cu": 1}     # kernels with bounded waits a file


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())


def kernels(name):
    """The bodies of a file's kernels (up to the brace in the first column) that allocate tensor memory."""
    out = [m.group(0) for m in re.finditer(r"__global__ void.*?\n}", source(name), flags=re.S)]
    return [k for k in out if "tmem_alloc(" in k and not re.search(r"\bdbg_\w+_kernel\(", k)]


def warp_parts(body):
    """Where whole warps work: what follows the branch that one thread of a warp takes (softmax, epilogue)."""
    start = max(body.rfind("regs_claim<"), body.rfind("else if (warp >= 4)"))
    return body[start:] if start >= 0 else body


@pytest.mark.parametrize("name", KERNELS)
def test_a_warp_gives_a_wait_up_as_a_whole(name):
    """A lane whose wait ran out must not leave while others go on into tcgen05.ld, a vote or a shuffle: there a wait
    answers for the whole warp, or only sets the lane's step count to 0, which the loop and the epilogue vote on."""
    found = kernels(name)
    assert len(found) == KERNELS[name]
    for body in found:
        part = warp_parts(body)
        assert re.search(r"tmem_ld\d+\(", part)
        counted = False
        for m in re.finditer(r"[^\n]*\bmbar_wait\([^\n]*", part):
            line = m.group(0)
            one_thread = "threadIdx.x == 0" in part[max(0, m.start() - 120):m.end()] or "&no_abort" in line
            counts = re.search(r"if \([^\n]*!mbar_wait\([^\n]*\)\) steps = 0;$", line) is not None
            assert "__all_sync" in line or one_thread or counts, line
            counted |= counts
        if counted:
            assert "; __all_sync(0xffffffffu, j < steps); ++j)" in part
            assert re.search(r"__all_sync\(0xffffffffu, steps == (nT|c)\)", part)


@pytest.mark.parametrize("name", KERNELS)
def test_what_is_in_flight_ends_before_the_block_does(name):
    """The waits for a block's own loads and products at its end keep the long limit: the test hooks take limits of a
    thousand clocks, which a load may exceed, and memory that a load still writes must not be given away."""
    for body in kernels(name):
        drains = re.findall(r"mbar_wait\([^\n]*&no_abort, (\w+)\)", body)
        assert len(drains) >= 2 and set(drains) == {"kDefaultTimeoutCycles"}, drains


@pytest.mark.parametrize("name,columns", [("sparse.cu", "AHEAD"), ("attention.cu", "OVER")])
def test_the_next_scores_wait_where_probabilities_lie_over_scores(name, columns):
    """BF16 with D = 128 keeps P in S's columns.  tcgen05 orders products only where they share accumulator and shape,
    so the product that reads P must be done before the next scores are written there; with D = 64, P lies beside S."""
    body = [k for k in kernels(name) if "issue_pv_bf16" in k][0]
    assert re.search(r"constexpr bool .*AHEAD = SC::AHEAD" if columns == "AHEAD" else r"constexpr bool OVER = D == 128;", body)
    after_pv = body[body.index("issue_pv_bf16"):]
    guard = re.search(r"if constexpr \((!AHEAD|OVER)\) \{(.*?)\n\s*\}", after_pv, flags=re.S)
    commit, wait = guard.group(2).index("mma_commit(&"), guard.group(2).index("mbar_wait(&")
    assert "p_read" in guard.group(2)[commit:commit + 25] and "p_read" in guard.group(2)[wait:wait + 25] and commit < wait
    next_scores = re.search(r"issue_(s|qk<D, false>)\(", after_pv)
    assert guard.start() + wait < next_scores.start()
    assert re.search(r"(AHEAD \? tmem \+ 384 \+ t \* 64 : d_s|OVER \? tmem \+ t \* 128 : tmem \+ 384 \+ t \* 64)", body)
