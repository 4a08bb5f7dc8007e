"""The 8-bit product's rings, step by step on the CPU.  Two groups take a ring's stages
in turn and wait on a barrier whose phases are told apart by a parity alone; copies may
land in any order that the slots allow.  The rule for the rings that a plan may have
(csrc/k_i8_matmul.cu, copies_in_order) is the one by which no wait passes early."""
import ctypes
import re
from pathlib import Path

import pytest

SOURCE = Path(__file__).parent.parent / "qwen3_dense_decoder_gb300" / "csrc" / "k_i8_matmul.cu"


def passes_early(ns, na, nb, stages=64):
    """Whether any order of events lets a group's wait for stage s pass while an earlier stage of its slot has not landed.

    A group waits for stage s knowing what it has waited for: copies of its own stages, and,
    from a free place of A (na) or B (nb, None where the group waits for none) at its last
    stage, that the products of all stages before that place's use are done, and with them
    their copies.  Whatever it does not know may not have happened yet."""
    for s in range(ns, stages):
        before = s - ns                                    # the stage that was in the slot
        if before % 2 == s % 2:
            continue                                       # the group's own
        last = s - 2
        done = max(last - na, last - nb if nb is not None else -1)
        if before > done:
            return True
    return False


def rule(cg, ns, na, nb):
    return ns % 2 == 0 or ns >= (min(na, nb) if cg == 1 else na) + 2


@pytest.mark.parametrize("cg", [1, 2])
def test_the_rule_is_that_no_wait_passes_early(cg):
    for ns in range(3, 9):
        for na in range(2, 5):
            for nb in range(3, 9):
                assert rule(cg, ns, na, nb) == (not passes_early(ns, na, nb if cg == 1 else None)), (ns, na, nb)


def test_every_plan_keeps_it():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()

    class Plan(ctypes.Structure):
        _fields_ = [(n, ctypes.c_int) for n in ("cg", "bn", "splits", "ns", "nb")]

    plan = q3.lib()._ZN2q37i8_planEiii
    plan.restype, plan.argtypes = Plan, [ctypes.c_int] * 3
    # the places of A by width, as the kernel has them
    widths = re.search(r"a_stages\(int bn\) \{ return bn > (\d+) \? 2 : bn > (\d+) \? 3 : MAX_NA; \}", SOURCE.read_text())
    two, three = map(int, widths.groups())
    seen = set()
    for m in (1, 300, 1024, 2560, 5120, 19456, 34816):
        for k in (1, 100, 1024, 2560, 4099, 9728, 17408, 131071):
            for t in (*range(17, 700), *range(700, 5000, 13)):
                p = plan(t, m, k)
                if p.cg:
                    seen.add((p.cg, p.bn, p.ns, p.nb))
    assert {cg for cg, *_ in seen} == {1, 2} and len(seen) > 10
    for cg, bn, ns, nb in seen:
        assert rule(cg, ns, 2 if bn > two else 3 if bn > three else 4, nb), (cg, bn, ns, nb)
