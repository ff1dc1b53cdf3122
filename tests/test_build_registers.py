"""Kernels that move registers between their warps (setmaxnreg) count on the number that a
thread is launched with: their launch refuses any other, and the build shows it first."""

import os
import re

import pytest

from block_speculative_decoding_ctx_gb300 import build as dbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    dbuild.build()


@pytest.mark.parametrize("unit", ["paged_attention_e2m1", "paged_attention_e2m1_rows"])
def test_registers_at_launch_are_what_the_split_counts_on(unit):
    with open(os.path.join(dbuild.CSRC, unit + ".cu")) as f:
        want = int(re.search(r"kRegsLaunch = (\d+)", f.read()).group(1))
    got = {k: v for k, v in dbuild.registers(unit).items() if unit + "_kernel" in k}
    assert len(got) == 2 and set(got.values()) == {want}, got


def test_every_kernel_with_such_a_split_is_looked_at():
    units = [n[:-3] for n in sorted(os.listdir(dbuild.CSRC)) if n.endswith(".cu")
             and re.search(r"reg_inc<|setmaxnreg", open(os.path.join(dbuild.CSRC, n)).read())]
    assert units == ["paged_attention_e2m1", "paged_attention_e2m1_rows"]


def test_the_log_is_read_as_ptxas_writes_it(tmp_path, monkeypatch):
    monkeypatch.setattr(dbuild, "BUILD", str(tmp_path))
    (tmp_path / "unit.ptxas").write_text("""ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_Za' for 'sm_103a'
ptxas info    : Function properties for _Za
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 88 registers, used 16 barriers
ptxas info    : Function properties for _Zb
    8 bytes stack frame, 4 bytes spill stores, 4 bytes spill loads
ptxas info    : Used 96 registers, used 4 barriers, 8 bytes cumulative stack size
""")
    assert dbuild.registers("unit") == {"_Za": 88, "_Zb": 96}
