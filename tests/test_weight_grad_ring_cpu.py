"""The ring of stages of the weight gradient's kernel, worked through on the CPU
from the constants in its source: who waits for which phase of a slot's codes."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "muon_polar_orthogonalized_b200", "csrc")


def geometry(wide):
    """(stages, groups, shared-memory bytes) of a tile geometry."""
    src = open(os.path.join(CSRC, "k_weight_grad.cu")).read()
    params = open(os.path.join(CSRC, "grad_params.cuh")).read()
    tiles = re.search(r"kWgTile\[2\] = \{\{(\d+), (\d+)\}, \{(\d+), (\d+)\}\}", params).groups()
    tn, tk = (int(v) for v in tiles[2 * wide:2 * wide + 2])
    stages = int(re.search(r"STAGES = WIDE \? (\d+) : (\d+);", src).group(1 if wide else 2))
    bk = int(re.search(r"WG_BK = (\d+);", src).group(1))
    warps = int(re.search(r"WG_WARPS = (\d+);", src).group(1))
    codes = tk // 2
    group_warps = bk * (codes // 16) // 32
    stage = tn // 256 * 2 * bk * 128 + codes // 64 * bk * 128 + codes * bk
    return stages, warps // group_warps, stages * stage + 2048


@pytest.mark.parametrize("wide", [0, 1])
def test_every_phase_of_a_slot_is_waited_for_by_its_group(wide):
    """A group knows of a slot's phases what it has waited for.  Its wait for use
    u of a slot passes as soon as the barrier's parity is not that of use u:
    with fewer than u completed uses of equal parity it could pass early, on use
    u - 2.  It cannot where it has waited for use u - 1 itself."""
    stages, groups, _ = geometry(wide)
    seen = {}   # (group, slot) -> uses waited for
    for s in range(8 * stages * groups):
        slot, use, group = s % stages, s // stages, s % groups
        assert seen.get((group, slot), 0) == use, f"group {group} comes to use {use} of slot {slot} from " \
                                                  f"use {seen.get((group, slot), 0) - 1}"
        seen[group, slot] = use + 1


@pytest.mark.parametrize("wide", [0, 1])
def test_the_ring_fits_in_shared_memory(wide):
    assert geometry(wide)[2] <= 227 * 1024
