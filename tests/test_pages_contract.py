"""Paged cache: what the sources and the host checks have to keep to (CPU only;
every library call made here with placeholder addresses fails a host check or
has nothing to do)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_bit_b200", "csrc")


def test_register_split_is_one_instruction_a_warpgroup():
    """PTX: all warps of a warpgroup execute the same setmaxnreg.  The many-row
    kernel's warps 12, 13 and 14, 15 have different roles and are one
    warpgroup, so the instruction stands ahead of the roles, once for each
    direction, under a condition on whole warpgroups."""
    with open(os.path.join(CSRC, "kvq_pages_tile.cuh")) as f:
        text = f.read()
    assert re.findall(r"setmaxnreg\.(inc|dec)", text) == ["inc", "dec"]
    split = re.search(r"if \(works\) \{\s*if \(warp < (\d+)\) asm volatile\(\"setmaxnreg\.inc[^;]*;\" ::\"n\"\(kSoftmaxRegs\)\);"
                      r"\s*else asm volatile\(\"setmaxnreg\.dec[^;]*;\" ::\"n\"\(kProducerRegs\)\);\s*\}", text)
    assert split and int(split.group(1)) % 4 == 0
    assert split.end() < text.index("warp >= 14")
