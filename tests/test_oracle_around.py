"""Pins of the oracles that stand around verification: drafts against probability
rows with given uniforms, 4-bit LM-head logits, and the pages of a cache."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import cache as OC
from oracle import probs as OP
from oracle import quant as OQ


def test_pick_is_the_inverse_of_the_running_sum():
    r = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [OP.pick(r, u)[0] for u in (0.0, 0.24, 0.25, 0.74, 0.75, 0.99)] == [1, 1, 3, 3, 4, 4]
    assert OP.pick(r, 1.0)[0] == 4 and OP.pick(r, math.nan)[0] == 4
    assert OP.pick(r, -1.0)[0] == 1
    assert OP.pick(np.zeros(3), 0.5)[0] == -1
    assert OP.pick(np.array([math.nan, -1.0, 2.0]), 0.9)[0] == 2


@pytest.mark.parametrize("rows", [True, False])
def test_first_token_follows_the_target(rows):
    """Speculative sampling's theorem: integrated over the uniforms (a grid of
    midpoints), the first emitted token has the target's law exactly."""
    p = np.array([[4, 2, 1, 1], [1, 1, 1, 1]]) / np.array([[8], [4]])
    q = np.array([[2, 2, 3, 1]]) / 8
    n = 32
    grid = [(i + 0.5) / n for i in range(n)]
    law = [Fraction(0)] * 4
    for d in range(4):
        weight = Fraction(int(q[0][d] * 8), 8) if rows else Fraction(int(d == 2))
        for u0 in grid:
            for u1 in grid:
                got = OP.verify(p, q if rows else None, [d], [u0, u1], 1)
                law[got.tokens[0]] += weight / (n * n)
    # acceptance steps lie on multiples of 1/8 over q; draws within a grid cell of a border
    for v in range(4):
        assert abs(float(law[v]) - p[0][v]) <= 2 / n


def test_bonus_and_ragged_rows():
    p = np.array([[0.5, 0.5], [1.0, 0.0], [0.0, 1.0]])
    assert OP.verify(p, None, [0, 0], [0.4, 0.0, 0.9], 2).tokens == [0, 0, 1]
    assert OP.verify(p, None, [0, 0], [0.4, 0.0, 0.9], 1).tokens == [0, 0]
    assert OP.verify(p, None, [0, 0], [0.4, 0.0, 0.9], -3).tokens == [1]
    assert OP.verify(p, None, [0, 0], [0.5, 0.0, 0.9], 2).tokens == [1]  # 0.5 < 0.5 fails


def test_quant_logits_by_hand():
    q = np.array([[0x10, 0x32, 0x54, 0x76] * 8], np.uint8)     # nibbles 0 .. 7, eight times
    assert OQ.unpack(q)[0, :8].tolist() == list(range(8))
    s = np.array([[0.5, 2.0]], np.float32)
    x = np.ones((1, 64), np.float32)
    # per group of 32: 4 * 28 - 32 z
    assert OQ.logits(x, q, s, None, 32)[0, 0] == 0.5 * (112 - 256) + 2.0 * (112 - 256)
    z = np.array([[0x31]], np.uint8)
    assert OQ.logits(x, q, s, z, 32)[0, 0] == 0.5 * (112 - 32) + 2.0 * (112 - 96)


def test_pages_through_a_step():
    rng = np.random.default_rng(0)
    c = OC.Pages(rng.standard_normal((2, 8, 4, 1, 2)), rows=3, max_blocks=4)
    assert c.reserve([6, 0, 0]) == [1, 1, 1] and c.tables[0] == [0, 1, -1, -1]
    c.lens[0] = 6
    assert c.fork([0, 0], [1, 2]) == [1, 1] and c.ref[:3] == [3, 3, 0] and c.lens == [6, 6, 6]
    before = c.pool[:, 1].copy()
    assert c.reserve([1, 5, 0]) == [1, 1, 1]
    assert c.tables[0] == [0, 2, -1, -1] and c.tables[1] == [0, 3, 4, -1]
    assert np.array_equal(c.pool[:, 2, :2], before[:, :2])
    assert np.array_equal(c.pool[:, 3, :2], before[:, :2])
    third = c.pool[:, 3, 3].copy(), c.pool[:, 4, 1].copy()
    # root at slot 6; accepted nodes 1 (slot 7) and 3 (slot 9, moved to slot 8)
    assert c.commit([0, 2], nodes=[[-1] * 5, [1, 3, -1, -1, -1]]) == [1, 1]
    assert c.lens[:2] == [7, 9] and np.array_equal(c.pool[:, 4, 0], third[1])
    assert np.array_equal(c.pool[:, 3, 3], third[0]) and c.consistent()
    c.truncate(new_len=[0, 5], rows=[2, 1])
    assert c.lens == [7, 5, 0] and c.tables[1] == [0, 3, -1, -1] and c.consistent()


def test_pages_refusals():
    c = OC.Pages(np.zeros((1, 3, 2, 1, 1)), rows=3, max_blocks=4)
    assert c.reserve([4, 4, 2]) == [1, 0, 0]        # one free page left, row 1 needs two
    assert c.reserve([4, -1, 2]) == [1, 0, 1] and c.consistent()
    assert c.fork([0, 0, 1], [1, 2, 0]) == [0, 1, 0]  # rows 0 and 1 are sources as well
    assert c.commit([0, 5, 9]) == [1, 0, 0]         # row 1 holds no pages; row 2's 9 lie behind them
    assert c.commit([1], nodes=[[2, -1, 0]], base=[6]) == [0]
    assert c.commit([2], nodes=[[2, 2, 0]], base=[0]) == [0]
    assert c.copy_pages([0, 1, 2, 9], [1, 2, 2, 0]) == [0, 0, 0, 0]


def test_commit_refuses_what_a_reserve_refused():
    """Rows that share the page they would write, and rows whose reserve's verdict is 0."""
    c = OC.Pages(np.arange(2 * 2 * 4, dtype=np.float64).reshape(2, 2, 4, 1, 1), rows=2, max_blocks=2)
    assert c.reserve([5, 0]) == [1, 1]
    assert c.commit([4, -1]) == [1, 0] and c.lens == [5, 0]
    assert c.fork([0], [1]) == [1] and c.ref == [2, 2]
    before = c.pool.copy()
    ok = c.reserve([3, 3])                          # a copy each of the last page: none is free
    assert ok == [0, 0]
    nodes = [[2, -1, -1]] * 2
    for reserved in (None, ok):                     # slot 7 to slot 6 of one page, for both
        assert c.commit([1, 1], nodes, reserved=reserved) == [0, 0]
        assert c.commit([0, 0], reserved=reserved) == [0, 0]
    assert c.lens == [5, 5] and np.array_equal(c.pool, before) and c.consistent()
    c.truncate(rows=[1])
    assert c.reserve([8, 0]) == [0, 1]              # 13 slots on 2 pages: behind the table
    assert c.commit([0, -1], reserved=[0, 1]) == [0, 0] and c.lens == [5, 0]
    assert c.commit([1, -1], nodes, reserved=[1, 1]) == [1, 0] and c.lens == [7, 0]
    assert np.array_equal(c.pool[:, 1, 2], before[:, 1, 3])


def test_commit_reads_counts_as_they_were():
    """A row that leaves a shared page does not make it another's own in the same call."""
    for rows in ([0, 1], [1, 0]):
        stays, leaves = rows
        c = OC.Pages(np.zeros((1, 3, 4, 1, 1)), rows=2, max_blocks=2)
        add, base = [0, 0], [0, 0]
        add[stays] = 5
        assert c.reserve(add) == [1, 1]
        c.lens[stays] = base[stays] = 5
        assert c.fork([stays], [leaves]) == [1] and c.ref == [2, 2, 0]
        add[stays], add[leaves] = 0, 1
        assert c.reserve(add, base=base) == [1, 1] and c.ref == [1, 2, 1]
        want = [0, 0]
        want[leaves] = 1
        assert c.commit([0, 0], base=base) == want
        assert c.ref == [1, 1, 1] and c.lens[stays] == 5 and c.lens[leaves] == 1 and c.consistent()
        assert c.commit([0, 0], base=base) == [1, 1]


def test_reserve_serves_rows_in_order():
    """Behind a row that does not fit none is served, also where it needs no page; a
    row refused by itself takes nothing from later ones."""
    c = OC.Pages(np.zeros((1, 5, 2, 1, 1)), rows=5, max_blocks=6)
    assert c.reserve([2, 4, 1, 0, 0]) == [1] * 5 and c.ref == [1, 1, 1, 1, 0]
    # row 0 needs two pages of one; the slots of rows 1 and 2 are their own; row 3 adds none
    assert c.reserve([6, 4, 2, 0, 1]) == [0, 0, 0, 0, 0]
    assert c.reserve([13, 4, 2, 0, 1]) == [0, 1, 1, 1, 1]   # behind the table, by itself
    assert c.reserve([-1, 4, 2, 0, 0], base=[0, 0, 0, 99, -1]) == [0, 1, 1, 1, 0]
    assert c.ref == [1] * 5 and c.consistent()
