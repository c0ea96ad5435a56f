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


def ends(rows, width, row, live, c, cols):
    """load_end's copies of one operand as (row of the stage, [row of the matrix or None for zeros]), and each box's first element."""
    out, at = [], []
    for i in range(0, cols, 64):
        if row + live >= 64:
            b, a0 = row + live - 64, 64 - live
            assert rows >= 64 and 0 <= b <= rows - 64 and 0 < a0 < 64        # the window lies in the matrix, and the box begins in it
            out.append((i, 0, [b + a if a < 64 else None for a in range(a0, a0 + 64)]))
            at.append((c + i, b + a0))
            continue
        r = 0
        while r + 16 <= live:
            out.append((i, r, list(range(row + r, row + r + 16))))
            at.append((c + i, row + r))
            r += 16
        while r < live:
            out.append((i, r, [row + r]))
            at.append((c + i, row + r))
            r += 1
        while r % 16:
            zero = (width + 7) // 8 * 8
            assert zero >= width and zero % 8 == 0                           # no column of the matrix, on a 16-byte boundary
            out.append((i, r, [None]))
            at.append((zero, row))
            r += 1
    return out, at


def test_the_end_of_a_group_is_copied_with_zeros():
    """The group's last rows, then zeros as far as products of 16 rows reach, each row once; the bytes that are waited for; and no box that
    begins before the matrix or below its last row."""
    src = source("moe_linear.cuh")
    for piece in ("return row + live >= kBoxRows;", "2 * (has_window(row, live) ? kBoxRows : (live + 15) / 16 * 16) * kBKBytes * (2 + cols / 64);",
                  "tma_3d<2>(dst + i * kBKBytes, windows, bar, c + i, kBoxRows - live, row + live - kBoxRows);",
                  "for (; r + 16 <= live; r += 16) tma_2d<2>(to + r * kBKBytes, &p.slab[operand], bar, c + i, row + r);",
                  "for (; r < live; ++r) tma_2d<2>(to + r * kBKBytes, &p.row[operand], bar, c + i, row + r);",
                  "for (; r % 16; ++r) tma_2d<2>(to + r * kBKBytes, &p.row[operand], bar, (width + 7) / 8 * 8, row);",
                  "dims[3] = {(cuuint64_t)width, kBoxRows, (cuuint64_t)(rows - kBoxRows + 1)}", "whole = kAcross && l.offsets && tl.sum % 16 ? nk - 1 : nk;",
                  "load_window(dst, &p.window[0], bar, f, kBM, row, live);",
                  "load_window(dst + kABlock, &p.window[1], bar, c, cols, row, live);", "load_rows(dst, p, 0, bar, f, kBM, p.l.N, row, live);",
                  "load_rows(dst + kABlock, p, 1, bar, c, cols, p.l.T, row, live);", "load_end(a, p, bar, wrow, xrow, tl.brows, row, live);"):
        assert piece in src, piece
    for rows in (1, 5, 15, 63, 64, 65, 200):
        for end in range(1, rows + 1):
            for live in range(1, min(64, end + 1)):
                if live % 16 == 0:
                    continue
                row, bytes_ = end - live, 0
                for cols in (128, 64):
                    copies, at = ends(rows, 997, row, live, 0, cols)
                    for i in range(0, cols, 64):
                        stage = {}
                        for j, r, got in copies:
                            if j == i:
                                for k, v in enumerate(got):
                                    assert r + k not in stage and r + k < 64
                                    stage[r + k] = v
                        assert [stage[k] for k in range(live)] == list(range(row, end))
                        assert all(stage[k] is None for k in range(live, (live + 15) // 16 * 16))
                        assert all(0 <= first < rows for _, first in at)
                    bytes_ += 128 * sum(len(got) for _, _, got in copies)
                assert 2 * bytes_ == 2 * (64 if end >= 64 else (live + 15) // 16 * 16) * 128 * (2 + 64 // 64)
