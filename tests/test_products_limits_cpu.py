"""The products' limits of dynamic shared memory, read from the source with the header that they share (no GPU here).

A limit belongs to the function: host threads that set different ones take it away from each other between setting and launch.  The
split kernels' is set at two places, before a launch and where their room on the GPU is asked for (capacity_of), which names them by a parameter."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "asynchronous_expert_execution_gb300", "csrc")
FILES = ("moe_linear.cu", "moe_linear_backward.cu", "moe_linear_blocks.cu")
SETS = r"cudaFuncSetAttribute\((\w+)(?:<[^()]*?>)?,\s*cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^)]*(?:\([^)]*\)[^)]*)?)\)"


def read(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def limits(header, src):
    """{kernel: the sizes that a translation unit's places set}: every kernel of a header belongs to the unit that includes it."""
    both = header + src
    asked = set(re.findall(r"capacity_of\((\w+)(?:<[^()]*?>)?,", both))
    found = {}
    for name, size in re.findall(SETS, both):
        for kernel in asked if name == "kernel" else (name,):
            found.setdefault(kernel, []).append(" ".join(size.split()))
    return found


def check(header, src):
    found = limits(header, src)
    for kernel, sizes in found.items():
        assert len(set(sizes)) == 1 and re.fullmatch(r"k[A-Z]\w*", sizes[0]), (kernel, sizes)
    return found


def test_every_place_sets_the_same_limit():
    header = read("moe_linear.cuh")
    assert header.count("cudaFuncSetAttribute(") == 1 and header.count("cudaFuncSetAttribute(kernel,") == 1       # capacity_of's
    for f in FILES:
        found = check(header, read(f))
        split = "linear_blocks_split_kernel" if f == "moe_linear_blocks.cu" else "linear_split_kernel"
        assert len(found[split]) == 2, (f, found)    # the launch's and capacity_of's
        assert len(found) >= 3 or f != "moe_linear_blocks.cu"


def test_another_limit_in_the_shared_header_is_seen():
    header = read("moe_linear.cuh")
    other = re.sub(r"(cudaFuncSetAttribute\(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, )kSplitSmem", r"\1kPairRing", header)
    assert other != header
    for f in FILES:
        try:
            check(other, read(f))
        except AssertionError:
            continue
        raise RuntimeError(f"{f}: two limits of one kernel went unseen")


def test_launches_ask_the_same_question_as_the_plans():
    """A split CTA takes a whole SM's ring only where the launch's clusters all find an SM a CTA: what the plan's cost took for granted."""
    for f, ask in (("moe_linear.cu", "split_capacity<kForward>"), ("moe_linear_backward.cu", "split_capacity<MODE>"), ("moe_linear_blocks.cu", "blocks_split_capacity")):
        assert f"tiles * splits <= {ask}(splits, sms)" in read(f), f
