"""The logit rules' kernels read a row's logits and grammar through buffers whose bounds stand in
for tests of their own, also where a wave's columns begin behind the row.  The bounds are compared
with a load's vector offset: a position in the scalar offset would not be sure to be held to them.
The kernels' own assembly shows where the positions stand (hipcc, no GPU)."""
from __future__ import annotations

import re
import subprocess

from vocab_selected_token_amd import build_lib


def test_no_position_of_a_load_stands_in_the_scalar_offset(tmp_path):
    out = tmp_path / "rlk_process.s"
    subprocess.run([build_lib.HIPCC, *build_lib.HIP_FLAGS, f"-I{build_lib.ROOT / 'include'}",
                    f"-I{build_lib.CSRC}", "--cuda-device-only", "-S",
                    str(build_lib.CSRC / "rlk_process.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    loads = re.findall(r"^\s*buffer_load_(\w+) v\S+, v\d+, s\[\d+:\d+\], (\S+) offen", text, re.M)
    assert len(loads) == text.count("buffer_load_")
    kinds = [kind for kind, _ in loads]
    # four kernels with four chunks a piece each: the first piece's and the next one's
    assert kinds.count("dwordx4") >= 4 * 4 * 2 and kinds.count("ubyte") >= 4 * 4 * 2
    assert {scalar for _, scalar in loads} == {"0"}
