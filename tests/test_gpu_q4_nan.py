"""A query with a NaN gives NaN in its own outputs and lse, whatever the length
of its row and the kernel that takes it, and changes nothing else."""
import pytest
import torch

from tests.test_gpu_q4 import Case

pytestmark = pytest.mark.gpu

NAN = float("nan")
# (seq, qo, Hkv): where the poisoned row lies
ROWS = {
    "within_one_warp": ([10, 70], [1, 1], 2),
    "cut_between_warps": ([200, 70], [1, 1], 2),
    "cut_between_ctas": ([9000, 70], [1, 1], 2),
    "three_queries": ([3000, 20], [3, 3], 2),
    "five_queries": ([3000, 20], [5, 5], 1),
    "five_queries_within_one_warp": ([9, 70], [5, 5], 2),
    "tile": ([900, 300], [40, 33], 8),
    "key_ranges": ([3000], [20], 2),
    "key_ranges_beside_decode_rows": ([9000, 900, 30], [40, 1, 1], 2),
}


@pytest.mark.parametrize("name", sorted(ROWS))
def test_a_query_with_nan_shows_in_its_own_rows_only(name):
    seq, qo, Hkv = ROWS[name]
    c = Case(seq, qo, Hkv, seed=len(name))
    want, want_lse = c.run()
    assert bool(torch.isfinite(want.float()).all()) and bool(torch.isfinite(want_lse).all())
    poisoned = torch.zeros(want_lse.shape, dtype=torch.bool, device=want.device)
    for tok, head in {(0, 1), (qo[0] // 2, 4 * Hkv - 1)}:
        c.dev["q"][tok, head, 77] = NAN
        poisoned[tok, head] = True
    out, lse = c.run()
    assert bool(torch.isnan(out[poisoned]).all())
    assert bool(torch.isnan(lse[poisoned]).all())
    assert torch.equal(out[~poisoned], want[~poisoned]) and torch.equal(lse[~poisoned], want_lse[~poisoned])
