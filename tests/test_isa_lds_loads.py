"""The post-build check for direct loads to LDS that stand too soon behind a
vector instruction's write of one of their scalar registers."""
import glob
import os

import pytest

from state_space_recurrence_amd import isa_check

LOAD = "s_mov_b32 m0, s48\ns_nop 0\nbuffer_load_dwordx4 v1, s[8:11], 0 offen lds"


@pytest.mark.parametrize("before, flagged", [
    ("v_readfirstlane_b32 s9, v3", True),
    ("v_readfirstlane_b32 s9, v3\ns_nop 1", True),
    ("v_readlane_b32 s11, v3, 2\nv_add_u32_e32 v1, 4, v1\ns_mov_b32 s2, 0", True),
    ("v_cmp_eq_u32_e64 s[10:11], v1, v2", True),
    # five wait states, other registers, scalar writes
    ("v_readfirstlane_b32 s9, v3\ns_nop 2", False),
    ("v_readfirstlane_b32 s9, v3\ns_mov_b32 s2, 0\ns_mov_b32 s3, 0\ns_mov_b32 s4, 0", False),
    ("v_readfirstlane_b32 s12, v3", False),
    ("s_mov_b32 s9, 0\nv_mov_b32_e32 v9, s9", False),
])
def test_rules(before, flagged):
    text = "_Zkern:\n" + "\n".join("\t" + line for line in f"{before}\n{LOAD}".splitlines()) + "\n"
    assert bool(isa_check.scan_lds_loads(text)) == flagged


def test_built_objects_are_clean():
    objs = glob.glob(os.path.join(os.path.dirname(isa_check.__file__), "_build", "scan_kernels.hip.o"))
    if not objs:
        pytest.skip("library not built")
    text = isa_check.disassemble(objs[0])
    assert text.count(" lds") > 100 and not isa_check.scan_lds_loads(text)
