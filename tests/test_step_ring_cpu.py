"""The ring of free blocks over many steps, without a GPU: whatever runs out,
ends or slides behind its window, every block stays in the ring or in one table.

`Loop` keeps what a serving loop keeps between its steps and makes each step by
a function with the oracle's arguments (the GPU tests give it the call)."""
import numpy as np
import pytest

from oracle import step


def oracle_step(new, cached, first, tables, ring, state, window, sinks, shared, n_tokens):
    return step.step_tables(new, cached, first, tables, ring, state, window, sinks, shared, n_tokens)


class Loop:
    def __init__(self, R, cap, max_blocks, window=0, sinks=0, n_tokens=None, seed=0, make=oracle_step):
        rng = np.random.default_rng(seed)
        self.cached, self.first = np.zeros(R, np.int32), np.zeros(R, np.int32)
        self.tables = np.full((R, max_blocks), -1, np.int32)
        self.ring, self.state = rng.permutation(cap).astype(np.int32), np.array([int(rng.integers(cap)), cap], np.int32)
        self.window, self.sinks, self.cap, self.n_tokens, self.make = window, sinks, cap, n_tokens, make

    def free(self):
        head, count = self.state
        return self.ring[(head + np.arange(count)) % self.cap].tolist()

    def held(self):
        """Blocks of the pages that the requests hold."""
        keep = -(-self.sinks // 16) if self.window else 0
        out = []
        for r, c in enumerate(self.cached):
            at = [j for j in range(-(-int(c) // 16)) if j < keep or j >= self.first[r]]
            out += [int(b) for b in self.tables[r, at] if b >= 0]
        return out

    def roll_back(self, r, c):
        """Request r keeps c tokens: the blocks of the pages behind them go back."""
        pages = -(-c // 16), -(-int(self.cached[r]) // 16)
        self.cached, self.ring, self.state = self.cached.copy(), self.ring.copy(), self.state.copy()
        for b in self.tables[r, pages[0]:pages[1]]:
            self.ring[self.state.sum() % self.cap] = b
            self.state[1] += 1
        self.cached[r] = c

    def step(self, new):
        """One step; the recorded errors.  Every block has to be somewhere, once."""
        new = np.asarray(new, np.int32)
        n = int(np.maximum(new, 0).sum()) if self.n_tokens is None else self.n_tokens
        before = self.cached.copy()
        got, errors = self.make(new, self.cached, self.first, self.tables, self.ring, self.state, self.window, self.sinks, 0, n)
        self.cached, self.first, self.state = got["seq_lens"], got["first_page"], got["free_state"]
        self.tables, self.ring, self.got = got["block_tables"], got["free_ring"], got
        assert sorted(self.free() + self.held()) == list(range(self.cap)), (before.tolist(), new.tolist())
        # what the tables and the slots say is one thing
        pos, slots, ind = got["positions"], got["slot_mapping"], got["qo_indptr"]
        for r in range(len(new)):
            for i in range(ind[r], ind[r + 1]):
                block = int(self.tables[r, pos[i] // 16])
                assert slots[i] == (block * 16 + pos[i] % 16 if block >= 0 else -1)
        return errors


def two_that_do_not_fit(make):
    """Four blocks, 64 tokens and 48: the second request gets none, ends, then
    the first does, and a third takes all four."""
    a = Loop(2, 4, 4, make=make)
    assert a.step([64, 48]) == {step.NO_BLOCKS}
    assert a.step([0, -1]) == set() and a.state[1] == 0
    assert a.step([-1, 0]) == set() and a.state[1] == 4
    assert a.step([0, 64]) == set() and a.state[1] == 0 and (a.tables[1] >= 0).all()


def a_prompt_larger_than_the_pool(make):
    a = Loop(3, 8, 20, make=make)
    assert a.step([160, 0, 0]) == {step.NO_BLOCKS}
    assert a.step([-1, 0, 0]) == set() and a.state[1] == 8 and a.cached.tolist() == [0, 0, 0]
    assert a.step([0, 100, 1]) == set() and a.state[1] == 0


def ends_beside_starts(make):
    """Ten blocks: a request that got seven of its nine pages ends while others
    start and end: more pages come back than there are places."""
    a = Loop(4, 10, 20, make=make)
    assert a.step([16, 20, 0, 0]) == set() and a.state[1] == 7
    assert a.step([0, 0, 144, 0]) == {step.NO_BLOCKS} and a.state[1] == 0
    assert a.step([-1, 0, 0, 0]) == set() and a.state[1] == 1
    assert a.step([0, -1, 0, 16]) == set() and a.state[1] == 2     # one granted, two back
    assert a.step([33, 0, -1, 0]) == {step.NO_BLOCKS}              # three wanted, two left; seven of nine back
    assert a.step([0, 0, 0, -1]) == set()
    assert a.step([-1, 0, 0, 0]) == set() and a.state[1] == 10


def tokens_of_a_page_without_a_block(make):
    """They are recorded in every step, and the page behind them is granted."""
    a = Loop(2, 2, 4, make=make)
    assert a.step([30, 1]) == {step.NO_BLOCKS}
    assert a.step([0, 1]) == {step.NO_BLOCKS} and a.got["slot_mapping"][:1].tolist() == [-1]
    assert a.step([-1, 0]) == set()
    assert a.step([0, 14]) == {step.NO_BLOCKS} and a.cached.tolist() == [0, 16]
    assert a.step([0, 1]) == set() and a.state[1] == 1             # its second page has one
    assert a.step([0, -1]) == set() and a.state[1] == 2


def pages_without_blocks_slide_behind_a_window(make):
    a = Loop(2, 5, 40, window=20, sinks=3, make=make)
    assert a.step([64, 40]) == {step.NO_BLOCKS}                    # 4 pages and 1 of 3
    for _ in range(60):
        a.step([1, 1])
    assert a.step([-1, -1]) == set() and sorted(a.free()) == list(range(5))


def drafts_are_refused(make):
    """Verify steps of five tokens of which some are kept, across page borders."""
    a = Loop(3, 40, 20, window=50, sinks=2, make=make)
    rng = np.random.default_rng(1)
    a.step([30, 1, 44])
    for _ in range(40):
        before = a.cached.copy()
        assert a.step([5, 5, 5]) == set()
        for r in range(3):
            a.roll_back(r, int(before[r] + rng.integers(1, 6)))
    a.step([-1, -1, -1])
    assert a.state[1] == 40


SEQUENCES = [two_that_do_not_fit, a_prompt_larger_than_the_pool, ends_beside_starts, tokens_of_a_page_without_a_block,
             pages_without_blocks_slide_behind_a_window, drafts_are_refused]


@pytest.mark.parametrize("sequence", SEQUENCES, ids=lambda f: f.__name__)
def test_no_block_is_lost_where_the_ring_runs_out(sequence):
    sequence(oracle_step)


def serve(loop, steps, seed, most=60):
    """A loop that ends a request that went without a block, and starts others in
    its place.  How many steps ran out, and how many tokens were made."""
    rng = np.random.default_rng(seed)
    R, short, made = len(loop.cached), 0, 0
    limit = loop.tables.shape[1] * 16
    ending = np.zeros(R, bool)
    for _ in range(steps):
        fresh = loop.cached == 0
        new = np.where(fresh, rng.integers(0, most + 1, R) * (rng.random(R) < 0.5), (rng.random(R) < 0.9).astype(int))
        new = np.where(~fresh & (ending | (rng.random(R) < 0.03) | (loop.cached + new > limit)), -1, new)
        if loop.n_tokens is not None and np.maximum(new, 0).sum() > loop.n_tokens:
            new = np.minimum(new, 1)
        errors = loop.step(new)
        assert errors <= {step.NO_BLOCKS}
        short += bool(errors)
        made += int(loop.got["qo_indptr"][-1])
        pages = -(-loop.cached // 16)
        ending = np.array([(loop.tables[r, max(int(pages[r]) - 1, 0):pages[r]] < 0).any() for r in range(R)])
    return short, made


# (behind a window of 16 a request holds two pages but in its first step)
@pytest.mark.parametrize("window,sinks,cap", [(0, 0, 30), (40, 5, 30), (16, 0, 18)])
def test_a_pool_that_is_too_small(window, sinks, cap):
    loop = Loop(12, cap, 12, window, sinks, seed=window)
    short, made = serve(loop, 300, window)
    assert short > 10 and made > 1000
    loop.step(np.where(loop.cached > 0, -1, 0))
    assert loop.state[1] == cap
