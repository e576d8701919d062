"""Compiler flags that sources rely on for their definitions (no GPU)."""
import os
import re

from qat_nvfp4_quantize_amd import build


def test_sources_of_the_block_encoder_are_built_without_contraction():
    """nvq_quant_block.h rounds products apart from sums; contraction would fuse them."""
    users = []
    for src in build.sources():
        with open(os.path.join(build.CSRC, src)) as f:
            if re.search(r'#include "nvq_quant_block\.h"', f.read()):
                users.append(src)
    assert users
    assert [s for s in users if "-ffp-contract=off" not in build.EXTRA.get(s, [])] == []
