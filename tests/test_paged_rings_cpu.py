"""Rings of the paged kernels, on the CPU: the waits of a streaming warp and of
the warps that consume its blocks, with the constants read out of the kernel
source, against copies that land as late as they can.

A wait on an mbarrier's phase parity returns as soon as the barrier is not in a
phase of that parity: the wait for use u of a slot also returns while use u - 1
has not landed. So whoever waits for a use must know that the one before it has.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "causal_sliding_window_rope_b200", "csrc")


def source(name):
    return open(os.path.join(CSRC, name)).read()


def choice(text, pattern):
    a, b = re.search(pattern, text).groups()
    return int(a), int(b)


def taken_early(stages, groups, late, blocks):
    """The first block that a group takes out of a slot before its copy has landed, or None; block n belongs to group
    n % groups, lies in slot n % stages, and the copy of block `late` lands only when nothing else can go on."""
    landed, full, empty = [False] * blocks, [0] * stages, [0] * stages  # phases completed
    issued, at = 0, list(range(groups))

    def land(n):
        landed[n] = True
        full[n % stages] += 1
    while True:
        moved = False
        if issued < blocks:
            use = issued // stages
            if use == 0 or empty[issued % stages] % 2 != (use - 1) % 2:
                if issued != late:
                    land(issued)
                issued += 1
                moved = True
        for g in range(groups):
            n = at[g]
            # (a block that is not issued yet: its slot's barrier is what the wait sees)
            if n < blocks and full[n % stages] % 2 != (n // stages) % 2:
                if not landed[n]:
                    return n
                empty[n % stages] += 1
                at[g] = n + groups
                moved = True
        if not moved:
            if late < issued and not landed[late]:
                land(late)
            else:
                break
    assert issued == blocks and min(at) >= blocks, "the ring stands still"
    return None


def test_the_model_sees_a_ring_whose_slots_change_hands():
    assert any(taken_early(10, 4, late, 60) is not None for late in range(30))
    assert all(taken_early(12, 4, late, 60) is None for late in range(60))


@pytest.mark.parametrize("wide_head", [False, True])
@pytest.mark.parametrize("many_groups", [False, True])
def test_weigh_rows_ring(wide_head, many_groups):
    """weigh_rows_kernel: its groups of warps take the blocks in turn."""
    text = source("paged_weigh.cuh")
    wide, narrow = choice(text, r"kStages = D == 128 \? (\d+) : (\d+);")
    many, few = choice(text, r"value = NT <= 2 \? (\d+) : (\d+);")
    stages, groups = wide if wide_head else narrow, many if many_groups else few
    for late in range(3 * stages):
        assert taken_early(stages, groups, late, 6 * stages) is None, late


def test_rows_ring():
    """rows_kernel: every warp waits for every block."""
    text = source("paged_rows.cuh")
    narrow, one, two = map(int, re.search(r"kStages = D == 64 \? (\d+) : \(MB == 1 \? (\d+) : (\d+)\);", text).groups())
    for stages in (narrow, one, two):
        for late in range(3 * stages):
            assert taken_early(stages, 1, late, 6 * stages) is None
