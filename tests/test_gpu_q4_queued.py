"""q4 calls queued behind one another on a stream, each launched while the one
before it may still run: every call sees what the calls before it wrote, and
no more."""
import numpy as np
import pytest
import torch

from paged_kv_decode_varlen_gb300 import workloads as W
from tests.test_gpu_q4 import DEV, _rows, bf16_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

# cached tokens, new tokens (in a page with cached ones), kv heads
SHAPES = {"small": ([45, 130, 7], [9, 40, 3], 2), "larger": ([1500, 700, 333, 90, 20], [30, 1, 64, 5, 12], 8)}


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_rounds_over_the_same_slots_see_their_own_rows(name, graph):
    cached, new, Hkv = SHAPES[name]
    rounds = 12
    rng = np.random.default_rng(7)
    lens = [a + b for a, b in zip(cached, new)]
    pages = [-(-L // 16) for L in lens]
    ids = rng.permutation(sum(pages) + 4).astype(np.int32)
    tables = np.full((len(lens), max(pages)), -1, np.int32)
    at = 0
    for r, p in enumerate(pages):
        tables[r, :p] = ids[at:at + p]
        at += p

    def slots(r, a, b):
        t = np.arange(a, b)
        return tables[r, t // 16].astype(np.int64) * 16 + t % 16

    old_slots = torch.from_numpy(np.concatenate([slots(r, 0, c) for r, c in enumerate(cached)])).to(DEV)
    new_slots = torch.from_numpy(np.concatenate([slots(r, c, L) for r, (c, L) in enumerate(zip(cached, lens))])).to(DEV)
    n = len(new_slots)
    kc, vc = B.new_q4_pool(len(ids), Hkv, DEV), B.new_q4_pool(len(ids), Hkv, DEV)
    base = bf16_dev(_rows(rng, len(old_slots), Hkv))
    B.pa_kv_append_q4(base, base.flip(0).contiguous(), old_slots, kc, vc)
    start = kc.clone(), vc.clone()
    tok = [bf16_dev(_rows(rng, n, Hkv)) for _ in range(rounds + 1)]  # round i: k = tok[i], v = tok[i + 1]
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    batches = []  # tile rows; rows of one query
    for qo in (new, [1] * len(lens)):
        q = bf16_dev(W.normal_bf16(rng, (sum(qo), 4 * Hkv, 128)))
        ind = np.concatenate([[0], np.cumsum(qo)]).astype(np.int32)
        batches.append((q, torch.from_numpy(ind).to(DEV), torch.from_numpy(ind)))
    tab = torch.from_numpy(tables).to(DEV)
    seq_host = torch.tensor(lens, dtype=torch.int32)
    ws = B.new_workspace(B.pa_attention_workspace_size(len(lens), n, 4 * Hkv, 128, max(lens)), DEV)

    def outputs():
        return [dict(before=[torch.zeros_like(tok[0]) for _ in range(2)], after=[torch.zeros_like(tok[0]) for _ in range(2)],
                     att=[torch.zeros_like(q) for q, _, _ in batches],
                     lse=[torch.zeros(q.shape[:2], device=DEV) for q, _, _ in batches]) for _ in range(rounds)]

    def run(outs, between):
        for i, o in enumerate(outs):
            B.pa_kv_read_q4(new_slots, kc, vc, k_out=o["before"][0], v_out=o["before"][1], workspace=ws)
            between()
            B.pa_kv_append_q4(tok[i], tok[i + 1], new_slots, kc, vc, workspace=ws)
            between()
            # the tile kernel and the read-back in turn come right after the append
            if i % 2 == 0:
                B.pa_kv_read_q4(new_slots, kc, vc, k_out=o["after"][0], v_out=o["after"][1], workspace=ws)
                between()
            for (q, ind, ind_host), out, lse in zip(batches, o["att"], o["lse"]):
                B.pa_attention_varlen_q4(q, kc, vc, tab, seq, ind, 0.088, seq_lens_host=seq_host,
                                         qo_indptr_host=ind_host, out=out, lse=lse, workspace=ws)
                between()
            if i % 2 == 1:
                B.pa_kv_read_q4(new_slots, kc, vc, k_out=o["after"][0], v_out=o["after"][1], workspace=ws)
                between()

    want = outputs()
    run(want, torch.cuda.synchronize)
    end = kc.clone(), vc.clone()
    kc.copy_(start[0])
    vc.copy_(start[1])
    got = outputs()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(got, lambda: None)
        kc.copy_(start[0])
        vc.copy_(start[1])
        torch.cuda.synchronize()
        g.replay()
    else:
        run(got, lambda: None)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    for i, (a, b) in enumerate(zip(want, got)):
        for key in a:
            for x, y in zip(a[key], b[key]):
                assert torch.equal(x, y), (i, key)
        if i > 0:  # the test itself: a round's rows differ from those before
            assert torch.equal(a["before"][0], want[i - 1]["after"][0])
            assert not torch.equal(a["after"][0], a["before"][0])
    assert torch.equal(kc, end[0]) and torch.equal(vc, end[1])


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("seq,qo", [([1500, 1200, 900, 800, 300, 700], [100, 1, 1, 1, 1, 1]),
                                    ([6000, 900, 30, 2000], [12, 5, 5, 5])], ids=["decode_rows", "key_ranges_and_verify_rows"])
def test_steps_rewrite_queries_tables_and_rows_in_place(seq, qo, graph):
    """Tile jobs and decode rows of one call, which run beside one another: a
    step's queries, block table and new rows are written over the last step's."""
    Hkv, steps = 2, 8
    rng = np.random.default_rng(9)
    pages = [-(-L // 16) for L in seq]
    total, blocks = sum(qo), sum(pages) + 9
    kc, vc = B.new_q4_pool(blocks, Hkv, DEV), B.new_q4_pool(blocks, Hkv, DEV)
    every = torch.arange(blocks * 16, device=DEV)
    B.pa_kv_append_q4(bf16_dev(_rows(rng, blocks * 16, Hkv)), bf16_dev(_rows(rng, blocks * 16, Hkv)), every, kc, vc)
    start = kc.clone(), vc.clone()
    per_step = []
    for _ in range(steps):
        ids = rng.permutation(blocks).astype(np.int32)
        tables = np.full((len(seq), max(pages)), -1, np.int32)
        at, slots = 0, []
        for r, (L, n, p) in enumerate(zip(seq, qo, pages)):
            tables[r, :p] = ids[at:at + p]
            at += p
            t = np.arange(L - n, L)
            slots.append(tables[r, t // 16].astype(np.int64) * 16 + t % 16)
        per_step.append([bf16_dev(W.normal_bf16(rng, (total, 4 * Hkv, 128))), torch.from_numpy(tables).to(DEV),
                         torch.from_numpy(np.concatenate(slots)).to(DEV), bf16_dev(_rows(rng, total, Hkv)),
                         bf16_dev(_rows(rng, total, Hkv))])
    q, tab, slot, k, v = (torch.empty_like(t) for t in per_step[0])
    lens = torch.tensor(seq, dtype=torch.int32)
    ind = torch.from_numpy(np.concatenate([[0], np.cumsum(qo)]).astype(np.int32))
    lens_dev, ind_dev = lens.to(DEV), ind.to(DEV)
    ws = B.new_workspace(B.pa_attention_workspace_size(len(seq), total, 4 * Hkv, 128, max(seq)), DEV)

    def run(outs, between):
        for new, (out, lse) in zip(per_step, outs):
            for dst, src in zip((q, tab, slot, k, v), new):
                dst.copy_(src)
            between()
            B.pa_kv_append_q4(k, v, slot, kc, vc, workspace=ws)
            between()
            B.pa_attention_varlen_q4(q, kc, vc, tab, lens_dev, ind_dev, 0.088, seq_lens_host=lens, qo_indptr_host=ind,
                                     out=out, lse=lse, workspace=ws)
            between()

    def outputs():
        return [(torch.zeros_like(q), torch.zeros(total, 4 * Hkv, device=DEV)) for _ in range(steps)]

    def rewind():
        kc.copy_(start[0])
        vc.copy_(start[1])
        torch.cuda.synchronize()

    want, got = outputs(), outputs()
    run(want, torch.cuda.synchronize)
    rewind()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(got, lambda: None)
        rewind()
        g.replay()
    else:
        run(got, lambda: None)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    for i, ((a, al), (b, bl)) in enumerate(zip(want, got)):
        assert torch.equal(a, b) and torch.equal(al, bl), i
    assert not torch.equal(want[0][0], want[1][0])
