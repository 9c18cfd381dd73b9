"""Rows cut between warps, CTAs and key ranges are put together by whichever
part comes last, in one order: a call repeated gives the same bits."""
import pytest
import torch

from tests.test_gpu_q4 import DEV, Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

BATCHES = {
    "between_warps": ([300 + 7 * i for i in range(60)], [1] * 60, 8),
    "between_warps_several_queries": ([400 + 11 * i for i in range(40)], [2 + i % 5 for i in range(40)], 8),
    "between_ctas": ([20000, 9000, 333], [1, 5, 3], 8),
    "tiles_and_ranges": ([6000, 900, 30, 2000], [40, 1, 1, 1], 2),
}


@pytest.mark.parametrize("name", sorted(BATCHES))
def test_a_call_repeated_gives_the_same_bits(name):
    seq, qo, Hkv = BATCHES[name]
    c = Case(seq, qo, Hkv, seed=len(name))
    ws = B.new_workspace(B.pa_attention_workspace_size(len(seq), sum(qo), 4 * Hkv, 128, max(seq)), DEV)
    want, want_lse = c.run(workspace=ws)
    c.check(want, want_lse, what=name)
    runs = [c.run(workspace=ws) for _ in range(100)]
    assert all(torch.equal(out, want) and torch.equal(lse, want_lse) for out, lse in runs)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
