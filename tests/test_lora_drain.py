"""The adapters' kernel for many rows after a wait that ran out: the products issued end before the block gives its tensor memory
back. A commit to a barrier tracks the products of the thread that executes it and no others', so every one of them, the
last one's too, belongs to the warp that issues the products. Read from the source (products that are still in flight when the
block leaves show in no run that ends well)."""
import os
import re

from tests._util import ROOT


def source():
    path = os.path.join(ROOT, "weight_quantized_gemm_gb300", "csrc", "lora_many.cuh")
    return re.sub(r"//[^\n]*", "", open(path).read())


def guard(src, at):
    """The condition on the warp of the innermost block around `at` that has one."""
    depth = 0
    for i in range(at, -1, -1):
        if src[i] == "}":
            depth += 1
        elif src[i] == "{":
            if depth:
                depth -= 1
                continue
            head = re.search(r"if \((warp == [^)]*?)\) $", src[:i])
            if head:
                return head.group(1)
    return None


def test_the_issuing_warp_commits():
    src = source()
    issued = [guard(src, m.start()) for m in re.finditer(r"\bmma_async<[\w:]+>\(tmem|\bmma_async<[\w:]+>\(d,", src)]
    commits = [guard(src, m.start()) for m in re.finditer(r"mma_commit<", src)]
    assert len(issued) == 2 and len(commits) == 3
    assert all(re.match(r"warp == S::kIssuer\b", g or "") for g in issued + commits), (issued, commits)


def test_the_last_commit_is_waited_for_with_the_full_bound_before_the_memory_is_released():
    src = source()
    last = src.rindex("mma_commit<")
    after = src[last:]
    wait, barrier, release = after.index("ptx::mbar_wait("), after.index("__syncthreads()"), after.index("tcgen05.dealloc")
    assert wait < barrier < release
    assert re.match(r"ptx::mbar_wait\([^,]*, 0, &never, p\.status\)", after[wait:])


def test_a_warp_is_whole_again_behind_a_wait_before_it_reads_tensor_memory():
    """A read of tensor memory is of the whole warp, whose lanes may leave a bounded wait one by one."""
    src = source()
    reads = [m.start() for m in re.finditer(r"gg::tmem_ld\(lanes", src)]
    assert len(reads) == 3
    for at in reads:
        before = src[:at]
        wait = max(before.rfind("wait(before"), before.rfind("wait(S::kStages"), before.rfind("auto empty"))
        between = before[before.rfind("\n", 0, wait):]
        assert "__syncwarp()" in between or "__syncthreads_or(fail)" in between
