"""What the kernels' sources may not hold: copies to the shared memory of several blocks at once.  The library is one file
that the processes of several GPUs load too, and its calls take pointers to any memory that the GPU can read; such a copy
is only for memory of the GPU itself."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_ssd_gb300", "csrc")


def test_no_bulk_copy_goes_to_several_blocks():
    sources = sorted(sum((glob.glob(os.path.join(CSRC, "*." + e)) for e in ("cu", "cuh", "h")), []))
    assert len(sources) > 20
    copies = 0
    for path in sources:
        with open(path) as fh:
            # (an instruction's text may go on in the next literal)
            text = re.sub(r'"\s*\n\s*"', "", fh.read())
        for instruction in re.findall(r"cp\.(?:reduce\.)?async\.bulk[^;]*;", text):
            copies += 1
            assert "multicast" not in instruction, (os.path.basename(path), instruction)
    assert copies >= 8
