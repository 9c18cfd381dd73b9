"""Infinities and NaN in values that some queries of a request see and others do
not.  A query that does not see them keeps its outputs: to the last bit in every
other dim, and in theirs within the bounds of test_gpu_window.py (such dims are
computed once more, in another order)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_window import DEV, Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

NOT_FINITE = [float("nan"), float("inf"), float("-inf")]

CASES = {
    "two": ([300, 70, 18], [2, 2, 2], 40, 3, 2),
    "verify": ([700, 512, 90, 31], [5, 4, 3, 6], 64, 4, 8),
    "verify_cut": ([3000, 2100], [5, 6], 1900, 0, 3),
    "verify_narrow": ([60, 33, 6], [6, 5, 4], 2, 1, 1),
    "seven_and_eight": ([300, 100], [7, 8], 50, 4, 2),
    "chunks": ([300, 500, 100], [40, 64, 33], 90, 4, 2),
    "chunk_of_many_jobs": ([900], [300], 128, 17, 2),
    "chunk_narrow": ([400], [100], 5, 1, 2),
    "whole_prompts": ([129, 250, 70], [129, 250, 70], 40, 20, 2),
    "sinks_in_the_chunk": ([90, 300], [90, 300], 17, 130, 1),
    "chunk_cut": ([6000], [100], 5000, 70, 1),
    "mixed": ([900, 40, 1, 2000, 513], [100, 1, 1, 4, 9], 300, 4, 2),
    "jobs_in_turn": ([400 + 7 * i for i in range(30)], [20 + 5 * i for i in range(30)], 200, 4, 8),
}


def planted(c, what, seed):
    """(row, position, kv head, dim) of values to replace: near both ends of what a
    row's queries see, where the queries differ."""
    rng = np.random.default_rng(seed)
    at = []
    for r, (L, n) in enumerate(zip(c.seq, c.qo)):
        p0 = int(L) - int(n)
        low = max(p0 - c.window + 1, 0)
        if n < 1:
            continue
        spots = {"last": [int(L) - 1], "diagonal": rng.integers(p0, L, 3).tolist(),
                 "first": [low, low + int(rng.integers(0, n))], "sinks": [min(max(c.sinks - 1, 0), int(L) - 1)]}
        for t in spots[what] if what != "all" else sum(spots.values(), []):
            if 0 <= t < L and (t < c.sinks or t >= low):
                for _ in range(3):
                    at.append((r, int(t), int(rng.integers(c.Hkv)), int(rng.integers(128))))
    return at


@pytest.mark.parametrize("what", ["last", "diagonal", "first", "sinks", "all"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_what_a_query_does_not_see_does_not_reach_it(name, what):
    seq, qo, window, sinks, Hkv = CASES[name]
    c = Case(seq, qo, window, sinks, Hkv, seed=len(name))
    want, want_lse = c.run()
    at = planted(c, what, len(name))
    dirty = torch.zeros_like(want, dtype=torch.bool)                  # outputs that see one
    near = dirty.clone()                                              # the same dims of all of the row's queries
    for i, (r, t, h, d) in enumerate(at):
        c.d["v"][int(c.tables[r, t // 16]), h, t % 16, d] = NOT_FINITE[i % 3]
        p = int(c.seq[r]) - int(c.qo[r]) + np.arange(c.qo[r])
        sees = (t <= p) & ((t < sinks) | (t > p - window))
        rows = torch.from_numpy(int(c.ind[r]) + np.flatnonzero(sees)).to(DEV)
        dirty[rows, 4 * h:4 * h + 4, d] = True
        near[int(c.ind[r]):int(c.ind[r + 1]), 4 * h:4 * h + 4, d] = True
    ws = c.workspace()
    for _ in range(2):
        out, lse = c.run(workspace=ws)
        assert torch.equal(lse, want_lse)
        assert torch.equal(out[~near], want[~near])
        assert not bool(torch.isfinite(out[dirty]).any()) and bool(dirty.any()) == bool(at)
        c.check(torch.where(dirty, want, out), lse)                   # (c.v is what the values were)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


@pytest.mark.parametrize("qo", [1, 2, 5, 9, 64])
def test_the_sign_of_an_infinity_and_two_that_cancel(qo):
    """A query that sees an infinity has it, one that sees both has a NaN."""
    inf = float("inf")
    c = Case([300], [qo], 100, 4, 1, seed=qo)

    def plant(t, dim, x):
        c.d["v"][int(c.tables[0, t // 16]), 0, t % 16, dim] = x

    plant(299, 5, inf)
    plant(299, 6, -inf)
    plant(298, 7, inf)
    plant(299, 7, -inf)
    out, _ = c.run()
    assert bool((out[-1, :, 5] == inf).all()) and bool((out[-1, :, 6] == -inf).all()) and bool(torch.isnan(out[-1, :, 7]).all())
    if qo > 1:
        assert bool((out[-2, :, 7] == inf).all()) and bool(torch.isfinite(out[-2, :, 5:7]).all())
    assert bool(torch.isfinite(out[:-2]).all())
    if qo == 1:
        again, _ = c.decode()
        assert torch.equal(again[..., :7], out[..., :7]) and bool(torch.isnan(again[:, :, 7]).all())
