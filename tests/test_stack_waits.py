"""What the kernels of the stacked blocks owe to the memory model and to a bounded wait that runs out, read from their
source: such runs cannot be brought about without a broken kernel, and what they must not do (leave while copies or peers'
stores are under way, read what only another lane has acquired) is a fault or a race."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parents[1] / "matrix_orthogonalising_optimizer_02_b200/csrc"


def body(kernel, file="stack_small.cu"):
    """The kernel's source, without comments."""
    text = re.sub(r"//[^\n]*", "", (CSRC / file).read_text())
    at = text.index(f"{kernel}(const __grid_constant__")
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError("unbalanced braces")


KERNELS = ["stack_small_kernel", "stack_small_grad_kernel"]


@pytest.mark.parametrize("kernel", KERNELS)
def test_no_cta_leaves_while_a_peer_may_store_into_it(kernel):
    """Behind the last iteration's stores every CTA of the cluster arrives at a barrier and waits for it before it frees
    its memory, whatever its own waits came to."""
    text = body(kernel)
    tail = text[text.rindex("st_async_v4("):text.rindex("tmem_dealloc(")]
    arrive = [m.start() for m in re.finditer(r"cluster_arrive\(\)|cluster_sum\(", tail)]
    wait = [m.start() for m in re.finditer(r"cluster_wait\(\)|cluster_sum\(", tail)]
    assert arrive and wait and wait[-1] >= arrive[-1]
    # neither depends on the iteration or on the CTA having given up
    for at in (arrive[-1], wait[-1]):
        line = tail[tail.rindex("\n", 0, at):at]
        assert "last" not in line and "abort" not in line


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_cta_that_gives_up_waits_for_what_is_under_way(kernel):
    """What is armed is counted, nothing is armed or multiplied after a wait has run out, and the count is waited for
    before the memory is freed."""
    text = body(kernel)
    end = text[:text.rindex("tmem_dealloc(")]
    assert "if (tid == 0 && *abort) drain_flight(" in end[end.rindex("slab_out_any"):]
    assert text.count("fly.arm(") == text.count("mbar_arrive_expect_tx(")
    assert "mbar_wait(" not in text            # through fly.wait() alone
    for m in re.finditer(r"tc_mma_bf16\(|mbar_arrive_expect_tx\(", text):
        before = text[:m.start()]
        guard = max(before.rfind("if (tid == 0 && fly.ok) {"), before.rfind("if (!fly.ok) return;"))
        assert guard >= 0 and guard > max(before.rfind("if (tid == 0) {"), before.rfind("__syncthreads();"))


def test_every_lane_of_the_epilogue_has_acquired_the_tile():
    """Lane 0 waits for the tile; the others read what it depends on only behind a barrier of the warp."""
    text = body("stack_chain_kernel", "stack_chain.cu")
    after = text[text.index("ti.n0 = __shfl_sync("):]
    first_read = min(after.index("cl.info["), after.index("prefetch_e(c_beg)"))
    assert "__syncwarp();" in after[:first_read]
