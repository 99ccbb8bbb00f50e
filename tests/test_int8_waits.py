"""CPU test of the streaming 8-bit product's hand-over in LDS, in the assembly that its source compiles to."""
import os
import re
import shutil
import subprocess

import pytest


def test_a_waves_sums_are_waited_for_before_the_barrier(tmp_path):
    """The barrier has no fence of its own.  Every store to LDS stands before the wait for its counter, the wait before
    the barrier, and the compiler is told of memory on both sides of the wait, so that it may not change that order."""
    from nvfp4_weight_streaming_amd import build as b
    if not shutil.which(b.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path / "int8.s"
    src = os.path.join(b.CSRC, "int8.hip")
    subprocess.run([b.HIPCC, *(f for f in b.flags_for(src) if f != "-fPIC"), "-S", "--cuda-device-only", src, "-o", str(out)],
                   check=True, capture_output=True)
    kernels = re.findall(r"^_ZN\w*int8_stream_kernel\w*:.*?s_endpgm\n(?=\t\.section)", out.read_text(), re.M | re.S)
    assert len(kernels) == 10
    for k in kernels:
        steps = re.findall(r"ds_write|#ASMSTART|lgkmcnt\(0\)|s_barrier|ds_read", k)
        barriers = [i for i, s in enumerate(steps) if s == "s_barrier"]
        assert barriers, k[:80]
        for i in barriers:
            before = steps[:i]
            last = max(j for j, s in enumerate(before) if s == "ds_write")
            assert [s for s in before[last + 1:] if s != "ds_read"] == ["#ASMSTART", "lgkmcnt(0)", "#ASMSTART"], (k[:80], before[last:])
            assert steps[i + 1] == "#ASMSTART"
