"""Host-side checks of the stateless operators beyond their refusals (no GPU here)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "asynchronous_expert_execution_gb300", "csrc")


def test_one_shared_memory_limit_a_kernel():
    """A kernel's limit of dynamic shared memory belongs to the function: host threads that set different ones take it
    away from each other between setting and launch.  Every place that sets an operator's limit gives the same constant."""
    limits = {}
    for f in ("moe_sort.cu", "moe_norm.cu", "moe_linear.cu"):
        src = open(os.path.join(CSRC, f)).read()
        local = dict(re.findall(r"const auto (\w+) = (\w+)<[^;]*>;", src))
        for name, size in re.findall(r"cudaFuncSetAttribute\((\w+)(?:<[^()]*?>)?,\s*cudaFuncAttributeMaxDynamicSharedMemorySize,\s*([^)]*(?:\([^)]*\)[^)]*)?)\)", src):
            limits.setdefault(local.get(name, name), set()).add(" ".join(size.split()))
    assert {"sort_experts_kernel", "rms_norm_backward_ring_kernel", "linear_split_kernel", "linear_pair_kernel"} <= set(limits)
    for name, sizes in limits.items():
        assert len(sizes) == 1, (name, sizes)
        assert re.fullmatch(r"(k[A-Z]\w*|\d+)( [*+] (k[A-Z]\w*|\d+))*", next(iter(sizes))), (name, sizes)
