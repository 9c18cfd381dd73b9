"""pa_step_tables over many steps in which the ring of free blocks runs out:
every step equals the oracle's, and no block is lost or given twice."""
import numpy as np
import pytest
import torch

from oracle import step
from tests.test_step_ring_cpu import SEQUENCES, Loop, serve

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

DEV = "cuda"
ORDER = ("seq_lens", "qo_indptr", "slot_mapping", "positions", "free_state", "first_page")


def caller(in_place, ws, pad=0):
    """The call as a step of a `Loop`, held to the oracle's; pad: rows of padding,
    which spread the launch over more CTAs."""
    def dev(a):
        return torch.from_numpy(np.array(a)).to(DEV)

    def call(new, cached, first, tables, ring, state, window, sinks, shared, n_tokens):
        n_tokens += pad
        want, errors = step.step_tables(new, cached, first, tables, ring, state, window, sinks, shared, n_tokens)
        d = [dev(x) for x in (new, cached, first, tables, ring, state)]
        kw = dict(seq_lens=d[1], first_page_out=d[2], free_state_out=d[5]) if in_place else {}
        out = B.pa_step_tables(d[0], d[1], d[3], d[4], d[5], n_tokens=n_tokens, window=window, sink_tokens=sinks,
                               shared_pages=shared, first_page=d[2], workspace=ws, **kw)
        torch.cuda.synchronize()
        err = B.pa_get_device_error(ws)
        assert (err in errors) if errors else err == 0
        ws[:4] = 0
        assert not ws.any()                      # nothing but the error word is left
        got = {k: t.cpu().numpy() for k, t in zip(ORDER, out)}
        got.update(block_tables=d[3].cpu().numpy(), free_ring=d[4].cpu().numpy())
        for k in ORDER + ("block_tables",):
            assert np.array_equal(got[k], want[k]), k
        head, count = got["free_state"]          # (what lies behind the ring's ids may be anything)
        live = (head + np.arange(count)) % len(ring)
        assert np.array_equal(got["free_ring"][live], want["free_ring"][live])
        return got, errors

    return call


FORMS = [(False, 0), (True, 0), (False, 5000), (True, 5000)]


@pytest.mark.parametrize("in_place,pad", FORMS)
@pytest.mark.parametrize("sequence", SEQUENCES, ids=lambda f: f.__name__)
def test_no_block_is_lost_where_the_ring_runs_out(sequence, in_place, pad):
    sequence(caller(in_place, B.new_workspace(256, DEV), pad))


@pytest.mark.parametrize("in_place,pad", FORMS)
@pytest.mark.parametrize("R,cap,window,sinks,steps", [(12, 30, 0, 0, 80), (12, 30, 40, 5, 80), (200, 330, 30, 3, 40),
                                                      (1100, 2500, 0, 0, 20), (1100, 1800, 40, 5, 20)])
def test_a_pool_that_is_too_small(R, cap, window, sinks, steps, in_place, pad):
    loop = Loop(R, cap, 12, window, sinks, seed=R + window, make=caller(in_place, B.new_workspace(256, DEV), pad))
    short, _ = serve(loop, steps, R)
    assert short > 3
    loop.step(np.where(loop.cached > 0, -1, 0))
    assert loop.state[1] == cap


@pytest.mark.parametrize("pad", [0, 5000])
def test_a_long_request_without_many_of_its_blocks_ends(pad):
    """Thousands of pages, most of them without a block, beside others that end and start."""
    make = caller(True, B.new_workspace(256, DEV), pad)
    loop = Loop(70, 3000, 8000, make=make)
    loop.step([100] * 66 + [0] * 4)
    assert loop.step([0] * 66 + [100_000, 0, 0, 0]) == {step.NO_BLOCKS}
    # (66 x 7 pages held, so 2538 of 6250 granted: none is left for those that start)
    assert loop.step([-1] * 30 + [1] * 36 + [-1, 50, 0, 20]) == {step.NO_BLOCKS}
    assert loop.step([0] * 30 + [-1] * 36 + [0, -1, 0, -1]) == set()
    assert loop.state[1] == 3000


@pytest.mark.parametrize("in_place,pad", FORMS)
@pytest.mark.parametrize("R", [1, 7, 60, 300, 1300])
def test_tables_and_rings_that_hold_anything(R, in_place, pad):
    """Entries and ids inside the pool and outside, lengths of all kinds, few places
    and many: the oracle's step, whatever it is."""
    make = caller(in_place, B.new_workspace(256, DEV), pad)
    rng = np.random.default_rng(R)
    done = short = 0
    for i in range(24):
        cap = int(rng.integers(1, [8, 4 * R, 40 * R][i % 3] + 2))
        cached = rng.integers(0, 150, R)
        new = np.where(rng.random(R) < 0.3, -1, rng.integers(0, 40, R) * (rng.random(R) < 0.5))
        tables = rng.integers(0, cap, (R, 12))
        tables[rng.random(tables.shape) < [0, 0.3, 0.9, 1][i % 4]] = -1
        tables[rng.random(tables.shape) < 0.02] = cap + 5
        ring = rng.integers(0, cap, cap)
        ring[rng.random(cap) < 0.02] = -3
        state = [int(rng.integers(cap)), int(rng.integers(0, cap + 1))]
        window, sinks = int(rng.choice([0, 20, 64])), int(rng.choice([0, 3, 40]))
        first = rng.integers(0, 4, R) if window else np.zeros(R)
        n = int(np.maximum(np.where(cached + new > 192, 0, new), 0).sum())
        i32 = [np.asarray(x, np.int32) for x in (new, cached, first, tables, ring, state)]
        got, errors = make(*i32, window, sinks, int(rng.choice([0, 0, 2])), n)
        short += step.NO_BLOCKS in errors
        done += got["qo_indptr"][-1] > 0 or not errors
    assert done > 2 and (R < 5 or short > 2)
