"""What orders the product kernels' shared memory between the CTAs of a cluster, read from the source (no GPU here)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "asynchronous_expert_execution_gb300", "csrc")


def source(name):
    """A file without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def kernel(src, name):
    """From a kernel's signature to the next kernel's or section's."""
    at = src.index(name + "(const __grid_constant__")
    end = re.search(r"\n__global__|\ntemplate <", src[at:])
    return src[at:at + end.start()] if end else src[at:]


def test_arrivals_over_the_cluster_say_so():
    """An arrive without qualifiers is a release over its own CTA only: one on another CTA's barrier has the cluster's scope, and one
    without an order is only for TMEM, whose fences stand around it."""
    ptx = source("moe_ptx.cuh")
    for op in re.findall(r'"(mbarrier\.arrive[^"]*)"', ptx):
        assert "shared::cluster" not in op or ".cluster.shared::cluster" in op, op
    for f in ("moe_linear.cuh", "moe_linear_backward.cu", "moe_linear_blocks.cu", "moe_linear.cu"):
        src = source(f)
        for m in re.finditer(r"mbar_arrive(\w*)\(([^;]*);", src):
            if "mapa" in m.group(2) or "tempty" in m.group(2):
                assert m.group(1) == "_relaxed" and "tempty" in m.group(2), (f, m.group(0))
                before = src[:m.start()]
                assert before.rindex("tc_before();") > before.rindex("tmem_ld") or "acc_done" in before[-400:], (f, m.group(0))


def test_waits_of_a_pair_have_the_clusters_scope():
    """The barriers of a pair's ring and accumulators hear of the other CTA's copies and products."""
    for f, name in (("moe_linear.cuh", "linear_pair_kernel"), ("moe_linear_blocks.cu", "linear_blocks_pair_kernel")):
        body = kernel(source(f), name)
        orders = {}
        for order, bar in re.findall(r"\bwait(<\w+>)?\(&s->(\w+)\[", body):
            orders.setdefault(bar, set()).add(order)
        assert orders["full"] == orders["empty"] == {"<kCluster>"} and orders["tfull"] == orders["tempty"] == {"<kTmem>"}, (name, orders)
    for f, name in (("moe_linear.cuh", "linear_split_kernel"), ("moe_linear_blocks.cu", "linear_blocks_split_kernel")):
        assert re.findall(r"\bwait(<\w+>)?\(&s->got", kernel(source(f), name)) == ["<kCluster>"], name      # the other ranks' partials


def test_a_pair_reads_what_copies_brought():
    """No thread writes operands that the other CTA's products read: the rows behind a group's end are copied as zeros."""
    body = kernel(source("moe_linear.cuh"), "linear_pair_kernel")
    assert "clear_rows" not in body and "load_end(" in body
    split = kernel(source("moe_linear.cuh"), "linear_split_kernel")
    assert "clear_rows" in split                     # there the products are the same CTA's, behind the fence


def test_the_end_of_a_group_is_copied_with_zeros():
    """load_end enters a window of 64 rows, whose first is `row`, at live - 64: what the copy brings, by its definition, is 64 - live rows of
    zeros and the group's `live` last, none of another's and none outside the matrix; the products take the rows from there on."""
    src = source("moe_linear.cuh")
    for piece in ("tma_3d<2>(dst + i * kBKBytes, m, bar, c + i, live - kBoxRows, row);", "dims[3] = {(cuuint64_t)width, kBoxRows, (cuuint64_t)rows}",
                  "n = (live + 15) / 16, first = CG == 2 ? kBoxRows / 16 - n : 0;"):
        assert piece in src, piece
    for rows in (1, 5, 63, 64, 65, 200):
        for end in range(1, rows + 1):
            for live in range(1, min(64, end + 1)):
                row = end - live
                got = [row + a if 0 <= a < 64 and 0 <= row < rows else None for a in range(live - 64, live)]
                assert got == [None] * (64 - live) + list(range(row, end)) and end <= rows
                n = (live + 15) // 16
                assert all(v is None for v in got[:64 - 16 * n]) and (n == 4 or live <= 48)
