"""How topk_kernel reads the rows of scores of a shared call, from its source: it may have written the row itself, through another
pointer, and a read through the kernel's __restrict__ argument would tell the compiler that nobody does.  (On a GPU that
shows as old scores, if at all.)"""
import re

from tests.test_pair_handover import body


def test_a_row_that_the_kernel_writes_is_read_through_the_pointer_that_it_writes():
    kernel = body("select.cu", "topk_kernel(const __half* __restrict__ scores")
    assert re.search(r"row = \(kShared \? ts\.scores : scores\) \+", kernel)
    plain = kernel[kernel.index("auto score_bits"):]
    plain = plain[plain.index("};"):]  # behind the one place that reads a score
    assert not re.search(r"\brow\[", plain)
    wide = [m.start() for m in re.finditer(r"\(row \+ c\)", plain)]
    assert len(wide) == 2  # eight at once: by ld.global, and by __ldg in calls whose rows another launch has written
    assert "if constexpr (kShared)" in plain[:wide[0]] and "ld.global" in plain[:wide[0]] and "__ldg" in plain[wide[0]:wide[1]]


def test_columns_between_the_prefix_and_the_own_cells_are_no_cells():
    # nobody writes them where a broken table keeps the score kernel from a prefix, and their cells may lie before the pool
    kernel = body("select.cu", "topk_kernel(const __half* __restrict__ scores")
    one = kernel[kernel.index("auto score_bits"):]
    one = one[:one.index("};")]
    assert one.index("if (in_gap(c)) return") < one.index("ld.global")
    wide = kernel[kernel.index("uint4 w[V / 8]"):kernel.index("w[m] = x;")]
    assert "in_gap(c + j)" in wide and "c + 8 > shared && c < shared + gap" in wide
