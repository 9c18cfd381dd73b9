"""q4 calls at the sizes from which other instantiations and further launches
take over: read-back of many rows, tile batches of many items, batches with
many verify rows."""
import numpy as np
import pytest
import torch

import oracle
from oracle import q4
from tests.test_gpu_q4 import DEV, Case, _rows, bf16_dev, bf16_host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B


@pytest.mark.parametrize("n,Hkv", [(8193, 8), (65541, 1), (21870, 3)])
def test_many_rows_are_written_and_read_back_bit_exact(n, Hkv):
    """More than 65,536 rows, in no whole number of CTAs; padding and a slot
    outside the pool among them."""
    assert n * Hkv > 65536 and n * Hkv % 64 != 0
    rng = np.random.default_rng(n)
    nb = n // 16 + 3
    k, v = _rows(rng, n, Hkv), _rows(rng, n, Hkv, "offset")
    slots = rng.permutation(nb * 16)[:n].astype(np.int64)
    slots[5::7] = -1
    kc, vc = B.new_q4_pool(nb, Hkv, DEV), B.new_q4_pool(nb, Hkv, DEV)
    ws = B.pa_kv_append_q4(bf16_dev(k), bf16_dev(v), torch.from_numpy(slots).to(DEV), kc, vc)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    asked = slots.copy()
    asked[n // 2] = nb * 16  # the first slot outside
    ko, vo = B.pa_kv_read_q4(torch.from_numpy(asked).to(DEV), kc, vc, workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    for rows, pool, got in ((k, kc, ko), (v, vc, vo)):
        codes, d, z = q4.quantize(rows)
        step = [np.repeat(oracle.bf16_to_f64(x), 32, -1) for x in (d, z)]
        want = q4.round_bf16(step[1] + step[0] * (1 + codes / 16))
        there = slots >= 0
        stored = q4.unpack(pool.cpu().numpy())[slots[there] // 16, :, slots[there] % 16]
        assert np.array_equal(stored, want[there])
        want[~there] = 0
        want[n // 2] = 0
        assert np.array_equal(bf16_host(got), want)


def _lens(seed, n, lo, hi):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi, n)]


TILES = {
    "more_than_160_items": (_lens(1, 200, 40, 90), _lens(2, 200, 7, 41), 2),
    "more_than_1536_items": (_lens(3, 1600, 12, 30), _lens(4, 1600, 7, 12), 1),
    "more_than_1536_items_beside_other_rows": (_lens(5, 1700, 12, 24), _lens(6, 1600, 7, 10) + _lens(7, 100, 0, 6), 1),
}


@pytest.mark.parametrize("name", sorted(TILES))
def test_tile_batches_of_many_items(name):
    seq, qo, Hkv = TILES[name]
    c = Case(seq, qo, Hkv, seed=len(name))
    ws = B.new_workspace(B.pa_attention_workspace_size(len(seq), sum(qo), 4 * Hkv, 128, max(seq)), DEV)
    B.pa_trace_enable(True)
    try:
        out, lse = c.run(workspace=ws)
        kinds = [k for k, _ in B.pa_trace_read()]
    finally:
        B.pa_trace_enable(False)
    c.check(out, lse, what=name)
    assert kinds.count("prefill") == (2 if "1536" in name else 1), kinds
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


VERIFY = {
    "more_than_128_rows_of_2_to_4": (_lens(11, 150, 4, 60), _lens(12, 150, 2, 5), 2),
    "more_than_128_rows_of_5_and_6": (_lens(13, 150, 6, 60), _lens(14, 150, 5, 7), 2),
    "both_and_single_queries": (_lens(15, 450, 6, 50), _lens(16, 150, 2, 5) + _lens(17, 150, 5, 7) + [1] * 150, 1),
    "more_than_1024_rows_of_3": (_lens(18, 1100, 3, 24), [3] * 1100, 1),
    "more_than_1024_rows_of_5_and_6": (_lens(19, 1100, 6, 24), _lens(20, 1100, 5, 7), 1),
}


@pytest.mark.parametrize("name", sorted(VERIFY))
def test_batches_of_many_verify_rows(name):
    seq, qo, Hkv = VERIFY[name]
    c = Case(seq, qo, Hkv, seed=len(name))
    ws = B.new_workspace(B.pa_attention_workspace_size(len(seq), sum(qo), 4 * Hkv, 128, max(seq)), DEV)
    B.pa_trace_enable(True)
    try:
        out, lse = c.run(workspace=ws)
        kinds = [k for k, _ in B.pa_trace_read()]
    finally:
        B.pa_trace_enable(False)
    c.check(out, lse, what=name)
    assert kinds == ["decode"] * (3 if name == "both_and_single_queries" else 2 if "1024" in name else 1), kinds
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
