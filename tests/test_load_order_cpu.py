"""Global loads of the kernels stay behind the wait for the kernel before them."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "reduction_pointwise_row_gb300", "csrc")


def test_every_global_load_is_ordered_and_coherent():
    """A kernel that begins with pdl_enter() may be placed while the kernel before it
    writes what it will read.  Assembly that is not volatile may be moved before the
    wait, and a read-only (.nc) load needs data that no one writes while the kernel
    lives: neither is used for global memory."""
    seen = 0
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for m in re.finditer(r"\basm\b(\s+volatile)?\s*\((.*?)\);", open(f).read(), flags=re.S):
            if "ld.global" not in m.group(2):
                continue
            seen += 1
            where = (os.path.basename(f), m.group(2)[:60])
            assert m.group(1), ("not volatile", *where)
            assert re.search(r':\s*"memory"\s*$', m.group(2)), ("no memory clobber", *where)
            assert ".nc" not in m.group(2), ("read-only load", *where)
    assert seen >= 7
