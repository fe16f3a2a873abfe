"""The linear layer's tile kernels as compiled: rows that go straight into LDS have arrived at the barrier behind which they
are read, whatever the lengths that lead there."""
import os

import pytest

from block_quantized_matrix_amd import bqm
from tests import _waits

STEP = """
  buffer_load_dwordx4 v1, s[0:3], s9 offen lds
  buffer_load_dwordx4 v1, s[0:3], s9 offen lds
{0}
<L{2}>:
  buffer_load_dwordx4 v[2:5], v6, s[4:7], s9 offen
  s_waitcnt vmcnt({1})
  s_barrier
  buffer_load_dwordx4 v1, s[0:3], s9 offen lds
  s_cbranch_scc1 L{2}
  s_endpgm"""


CODES = "buffer_load_dwordx4 v[8:11], v6, s[4:7], s9 offen"


@pytest.mark.parametrize("between,wait,under_way", [
    ("", 2, 0), ("", 3, 1),                                      # the first round has two operations behind the first rows
    (CODES, 3, 0), (CODES, 4, 1),                                # three, as the others have
    ("s_waitcnt vmcnt(0)", 3, 0), ("s_waitcnt vmcnt(0)", 4, 1)])  # there they have arrived, on the others three again
def test_reader_follows_every_path(between, wait, under_way):
    ins, before = _waits.parse(STEP.format(between, wait, 7).splitlines())
    b = ins.index("s_barrier")
    assert _waits.stage_behind(ins, b) == 1
    assert _waits.outstanding(ins, before, b, 1) == under_way


def test_rows_have_arrived_where_they_are_read(tmp_path):
    """At a barrier in the tile kernels all rows have to be in LDS but those of one stage, as many loads as are issued
    right behind it."""
    if not os.path.exists(_waits.OBJDUMP):
        pytest.skip("llvm-objdump is not installed")
    kernels = {n: v for n, v in _waits.disassemble(bqm.LIB_PATH, str(tmp_path)).items() if "k_linear_tiles" in n}
    assert len(kernels) >= 36  # three formats by five tiles for two types and two for the third
    early, staged = [], 0
    for name, lines in kernels.items():
        ins, before = _waits.parse(lines)
        for b, t in enumerate(ins):
            if t == "s_barrier":
                newest = _waits.stage_behind(ins, b)
                staged += newest > 0
                n = _waits.outstanding(ins, before, b, newest)
                if n:
                    early.append(f"{name}: barrier at instruction {b}, {n} operations since rows that are read behind it")
    assert staged >= 7 * len(kernels)  # the seven steps of each pipeline
    assert not early, "\n".join(early)
