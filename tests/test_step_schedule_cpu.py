"""Attention over trees with many rows: how a block's roles wait for one another,
replayed without a GPU (step_schedule)."""

import random

import pytest

import step_schedule as sched


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("case", sorted(sched.CASES))
def test_every_role_ends(case, whole):
    """Every block of a call that gives some of them a long run of single tiles behind a shared piece."""
    blocks = sched.pieces(*sched.CASES[case], whole=whole)
    runs = [sched.run_of_single_tiles(b) for b in blocks]
    assert max(runs) > sched.RING
    r = random.Random(len(case))
    for slots in (3, 4):
        for b in blocks:
            assert sched.Block(b, slots).run(r) == []


@pytest.mark.parametrize("case", sorted(sched.CASES))
def test_looking_for_the_next_piece_first_would_wait_for_ever(case):
    """The order that these calls are there for: a warpgroup that passes over more pieces than the ring holds before
    it hands its half of a shared one over, which the other waits for."""
    r = random.Random(len(case))
    for b in sched.pieces(*sched.CASES[case]):
        stuck = sched.Block(b, 4, search_first=True).run(r)
        assert bool(stuck) == (sched.run_of_single_tiles(b) > sched.RING)


def test_pieces_of_any_kind_in_any_order():
    r = random.Random(6)
    for _ in range(400):
        block = [(r.choice([1, 1, 1, 2, 3, 5]), r.choice([8, 100, 128, 129, 256])) for _ in range(r.randint(1, 30))]
        for slots in (3, 4):
            assert sched.Block(block, slots).run(r) == []


def test_pieces_are_the_items_whole_or_cut():
    for case in sched.CASES.values():
        line = sched.items(*case)
        total = sum(n for n, _ in line)
        whole, cut = (sched.pieces(*case, whole=w) for w in (True, False))
        assert [p for b in whole for p in b] == line
        assert sum(n for b in cut for n, _ in b) == total
        sizes = [sum(n for n, _ in b) for b in cut]
        assert max(sizes) - min(sizes) <= 1
