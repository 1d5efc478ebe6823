"""Dynamic shared memory that is read by vectors says its own alignment, or aligns itself: behind a kernel's static shared
memory the type's alignment alone holds."""
from __future__ import annotations

import glob
import os
import re

from jagged_attention_recommender_gb300 import build as gbuild


def test_dynamic_shared_memory_is_aligned_for_vectors():
    seen = 0
    for path in sorted(glob.glob(os.path.join(gbuild.CSRC, "*.cu*"))):
        text = open(path).read()
        for m in re.finditer(r"extern __shared__ (?:__align__\((\d+)\) )?\w+ (\w+)\[\];", text):
            seen += 1
            by_hand = "smem_u32(%s) & 1023" % m.group(2) in text[m.end():m.end() + 200]
            assert by_hand or int(m.group(1) or 0) >= 16, (os.path.basename(path), m.group(0))
        assert text.count("extern __shared__") == len(re.findall(r"extern __shared__ (?:__align__\(\d+\) )?\w+ \w+\[\];", text))
    assert seen >= 10
