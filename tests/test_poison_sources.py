"""Every kernel's LDS is filled in the debug copy of the library: each array has its macro right behind
it.  Reads the sources; no GPU."""
import glob
import os
import re

import dense_fp16_gemm_f16_amd.build as build

# the row plan's kernels, which clear all of their LDS before they use it, and the rate probe,
# which is not part of the library
ELSEWHERE = {"seg_group.hip": 2, "mfma_ceiling.hip": 2}


def test_every_lds_array_is_poisoned():
    found = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.h")) + glob.glob(os.path.join(build.CSRC, "*.hip"))):
        with open(path) as f:
            lines = f.read().splitlines()
        arrays = [(i, m[1]) for i, line in enumerate(lines)
                  if (m := re.match(r"\s*(?:extern )?__shared__ .*?(\w+)\[[^()]*\];?", re.sub(r"__attribute__\(\(.*?\)\)\)", "", line)))]
        name = os.path.basename(path)
        if name in ELSEWHERE:
            assert len(arrays) == ELSEWHERE[name], name
            continue
        for i, array in arrays:
            found += 1
            assert any(re.search(rf"GEMM_POISON_LDS(_BYTES)?\({array}\b", x) for x in lines[i + 1:i + 4]), (name, i + 1, array)
    assert found >= 20
