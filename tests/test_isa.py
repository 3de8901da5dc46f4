"""What the hardware asks of the instruction stream and the compiler does not see, because the instruction stands in
an asm statement: checked in the built library's own code."""
import os
import re

import pytest

import combine_moe_get_amd as mg
from tests import _isa

pytestmark = pytest.mark.skipif(not os.path.exists(_isa.OBJDUMP) or not os.path.exists(mg.LIB_PATH),
                                reason="needs llvm-objdump and the built library")


@pytest.fixture(scope="module")
def kernels():
    return _isa.kernels()


def _sregs(operand):
    """Numbers of the scalar registers that an operand names: s5, s[4:7]."""
    m = re.fullmatch(r"s(\d+)|s\[(\d+):(\d+)\]", operand)
    if not m:
        return set()
    return {int(m.group(1))} if m.group(1) else set(range(int(m.group(2)), int(m.group(3)) + 1))


def _vector_writes(ins):
    """Scalar registers that a vector instruction writes: its first operand; of a carry, the second."""
    op, _, rest = ins.partition(" ")
    if not op.startswith("v_"):
        return set()
    names = [o.strip() for o in rest.split(",")]
    return _sregs(names[0]) | (_sregs(names[1]) if ("_co_" in op or "div_scale" in op) and len(names) > 1 else set())


def _wait_states(ins):
    return int(ins.split()[1], 0) + 1 if ins.startswith("s_nop") else 1


def distance(body, at):
    """Wait states before the memory instruction body[at] back to a vector instruction that writes one of its scalar
    registers, or to where that is no longer known (a label, the kernel's start); at most 5."""
    need = set().union(*(_sregs(o.strip()) for o in re.split(r"[ ,]+", body[at])[1:]))
    states = 0
    for ins in reversed(body[:at]):
        if states >= 5 or ins.endswith(":") or _vector_writes(ins) & need:
            return min(states, 5)
        states += _wait_states(ins)
    return states


def test_distance():
    load = "buffer_load_dwordx4 v0, s[24:27], s72 offen lds"
    near = ["v_readfirstlane_b32 s24, v0", "s_mov_b32 s27, 0", "s_add_u32 m0, s73, 0", "s_nop 0", load]
    assert distance(near, 4) == 3
    assert distance(["v_add_co_u32_e64 v1, s[72:73], v2, v3", "s_nop 3", load], 2) == 4
    assert distance(["v_readfirstlane_b32 s28, v0", "s_nop 7", load], 2) == 5
    assert distance(["v_readfirstlane_b32 s24, v0", "L3:", "s_nop 2", load], 3) == 3
    assert distance(["v_cmp_gt_i32_e64 s[26:27], v0, v1", "s_nop 1", "s_nop 1", "s_nop 0", load], 4) == 5


def test_loads_to_lds_keep_their_distance_from_the_descriptors_writes(kernels):
    """A vector instruction's write of a scalar register needs five wait states before a memory instruction reads it."""
    near, loads = [], 0
    for name, body in kernels.items():
        for i, ins in enumerate(body):
            if ins.startswith("buffer_load") and ins.endswith(" lds"):
                loads += 1
                if distance(body, i) < 5:
                    near.append(f"{name}: {distance(body, i)}")
    assert loads > 0
    assert not near, f"{len(near)} of {loads} loads, in {len({n.rsplit(':', 1)[0] for n in near})} kernels: {near[:4]}"


def test_m0_is_the_loads_own(kernels):
    """M0 holds the LDS address of the loads, written by each for itself: nothing else in such a kernel keeps a value
    there or reads one."""
    for name, body in kernels.items():
        if not any(ins.startswith("buffer_load") and ins.endswith(" lds") for ins in body):
            continue
        uses = [i for i, ins in enumerate(body) if re.search(r"\bm0\b", ins)]
        for i in uses:
            assert body[i].startswith("s_add_u32 m0,") and "m0" not in body[i].split(",", 1)[1], (name, body[i])
            assert any(ins.startswith("buffer_load") for ins in body[i + 1:i + 3]), (name, body[i:i + 3])
