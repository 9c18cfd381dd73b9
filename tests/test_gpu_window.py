"""pa_attention_varlen_window and pa_decode_window through the C ABI against
the definition in 64 bits.

Whatever no query of a request sees is not a number here: slots behind the last
token, tokens behind the window, blocks of no table; pages without a visible
token have no block.

Bounds, as for the other attention calls.  Scores: 128 products of bf16 numbers
are exact in binary32; summing them and scaling rounds each at most 2^-24 relative
some 136 times, so a score is off by at most DS = 2^-16 sm_scale max_t sum_d |q_d
k_td|.  Then lse is off by at most DS plus a few roundings of its own, and every
probability by a factor exp(2 DS).  The weights of rows with more than two queries
are rounded to bf16 (2^-8 each) before they meet V, the others carry 16 bits; an
output is rounded once to bf16.  With A = sum_t p_t |v_t|:
  |out - ref| <= 2^-8 |ref| + (w + 4 DS + 2^-14) A,  w = 2^-8 or 2^-15.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import step
from paged_kv_decode_varlen_gb300 import workloads as W
from tests.util import bf16_dev, bf16_host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

DEV = "cuda"


class Case:
    def __init__(self, seq, qo, window, sinks=0, Hkv=2, seed=0, scale=1 / np.sqrt(128), spare=3):
        rng = np.random.default_rng(seed)
        R = len(seq)
        self.seq, self.qo = np.asarray(seq, np.int32), np.asarray(qo, np.int32)
        self.ind = np.concatenate([[0], np.cumsum(self.qo)]).astype(np.int32)
        self.window, self.sinks, self.Hkv, self.scale = window, sinks, Hkv, float(np.float32(scale))
        pages = -(-self.seq // 16)
        self.tables = np.full((R, max(1, int(pages.max(initial=1)))), -1, np.int32)
        seen = []                                    # (row, token) that some query of the row sees
        for r in range(R):
            if qo[r]:
                t = np.arange(seq[r])
                seen.append((r, t[(t < sinks) | (t > seq[r] - qo[r] - window)]))
        need = sorted({(r, int(j)) for r, t in seen for j in t // 16})
        nb = len(need) + spare
        perm = rng.permutation(nb)
        for i, (r, j) in enumerate(need):
            self.tables[r, j] = perm[i]
        self.k = np.full((nb, Hkv, 16, 128), 0x7fc0, np.uint16)
        self.v = self.k.copy()
        self.v[:, :, ::3] = 0x7f80                   # infinities too
        for r, t in seen:
            at = (self.tables[r, t // 16], slice(None), t % 16)
            self.k[at], self.v[at] = W.normal_bf16(rng, (len(t), Hkv, 128)), W.normal_bf16(rng, (len(t), Hkv, 128))
        self.q = W.normal_bf16(rng, (int(self.ind[-1]), 4 * Hkv, 128))
        self.d = dict(q=bf16_dev(self.q), k=bf16_dev(self.k), v=bf16_dev(self.v), tables=torch.from_numpy(self.tables).to(DEV),
                      seq=torch.from_numpy(self.seq).to(DEV), ind=torch.from_numpy(self.ind).to(DEV))

    def workspace(self):
        return B.new_workspace(B.pa_window_workspace_size(len(self.seq), len(self.q), 4 * self.Hkv, 128, self.window,
                                                          self.sinks), DEV)

    def run(self, **kw):
        d = self.d
        return B.pa_attention_varlen_window(d["q"], d["k"], d["v"], d["tables"], d["seq"], d["ind"], self.scale, self.window,
                                            self.sinks, seq_lens_host=torch.from_numpy(self.seq),
                                            qo_indptr_host=torch.from_numpy(self.ind), return_lse=True, **kw)

    def decode(self, **kw):
        """The batch's rows of one query through the call that plans on the device."""
        d = self.d
        return B.pa_decode_window(d["q"], d["k"], d["v"], d["tables"], d["seq"], self.scale, self.window, self.sinks,
                                  return_lse=True, **kw)

    def check(self, out, lse, what="", rows=None):
        ref, ref_lse, weight = step.attention_window(self.q, self.k, self.v, self.tables, self.seq, self.ind, self.scale,
                                                     self.window, self.sinks)
        kmax = np.nanmax(np.abs(oracle.bf16_to_f64(self.k)), initial=0)
        ds = 2.0 ** -16 * abs(self.scale) * kmax * np.abs(oracle.bf16_to_f64(self.q)).sum(-1)
        w = np.where(np.repeat(self.qo, self.qo) > 2, 2.0 ** -8, 2.0 ** -15)
        tol = 2.0 ** -8 * np.abs(ref) + (w[:, None] + 4 * ds + 2.0 ** -14)[..., None] * weight
        got = oracle.bf16_to_f64(bf16_host(out))
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5].tolist(),
                               float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-30))))
        lerr = np.abs(lse.cpu().double().numpy() - ref_lse)
        assert np.all(lerr <= ds + 2.0 ** -20 * (1 + np.abs(ref_lse))), (what, float(lerr.max()))


def rand(seed, n, lo, hi):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi + 1, n)]


DECODE = {
    "one_token": ([1], 1, 0, 1),
    "window_of_one": ([1, 16, 17, 40], 1, 0, 2),
    "window_of_one_and_sinks": ([1, 2, 16, 17, 40], 1, 3, 2),
    "page_edges": (list(range(30, 68)), 17, 0, 1),
    "page_edges_sinks": (list(range(30, 68)), 16, 16, 1),
    "window_meets_sinks": (list(range(1, 60)), 20, 18, 1),
    "sinks_alone_reach": ([100, 50, 7], 2, 200, 2),
    "wide": ([100, 700, 16], 10 ** 6, 0, 2),
    "widest": ([100, 700, 16], 2 ** 31 - 1, 2 ** 31 - 1, 2),
    "three_heads": ([1000, 70, 300], 128, 4, 3),
    "twelve_heads": ([129, 640, 1, 500], 100, 4, 12),
    "eight_heads": ([17, 100, 2560, 513], 256, 4, 8),
    "long_and_short": ([9000, 1, 40, 2100, 16], 4000, 5, 2),
    "one_long": ([20000], 16000, 70, 1),
    "many_rows": (rand(4, 300, 1, 200), 50, 4, 1),
    "rows_over_one_launch": (rand(5, 1100, 1, 60), 20, 1, 1),
    "as_the_batch": (rand(6, 64, 300, 3000), 512, 4, 8),
}


@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode_rows(name):
    seq, window, sinks, Hkv = DECODE[name]
    c = Case(seq, [1] * len(seq), window, sinks, Hkv, seed=len(name))
    ws = c.workspace()
    c.check(*c.run(workspace=ws), what=name)
    c.check(*c.decode(workspace=ws), what=name + ", planned on the device")
    c.check(*c.run(workspace=ws), what=name + ", the workspace again")
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


MANY = {
    "two_queries": ([2, 300, 17, 16], [2, 2, 2, 2], 30, 0, 3),
    "verify": ([700, 512, 90, 31], [5, 5, 5, 5], 64, 4, 8),
    "three_to_nine": ([40, 333, 16, 17, 90, 3000, 9], [3, 4, 5, 6, 7, 8, 9], 50, 3, 2),
    "eight_of_few": ([8, 9, 24, 100], [8, 8, 8, 8], 4, 1, 2),
    "whole_prompts": ([1, 16, 17, 33, 129, 250], [1, 16, 17, 33, 129, 250], 40, 0, 2),
    "whole_prompts_sinks": ([16, 17, 33, 129, 250], [16, 17, 33, 129, 250], 40, 20, 2),
    "chunk_late": ([1500, 600], [70, 33], 200, 4, 1),
    "chunk_narrow": ([500, 600], [170, 133], 5, 1, 2),
    "chunk_wide": ([500, 600], [170, 133], 10 ** 6, 0, 2),
    "chunk_tile_edges": ([128, 129, 160, 257, 96], [32, 33, 31, 64, 65], 64, 0, 1),
    "window_is_a_tile": ([400, 513, 640], [64, 65, 100], 128, 128, 1),
    "sinks_in_the_chunk": ([90, 300], [90, 300], 17, 130, 1),
    "mixed": ([900, 40, 1, 2000, 513, 77], [100, 1, 1, 1, 7, 0], 300, 4, 2),
    "idle_rows": ([50, 0, 30, 70, 9], [0, 0, 3, 0, 1], 10, 0, 2),
    "jobs_in_turn": (rand(6, 40, 7, 400), rand(7, 40, 1, 100), 90, 4, 8),
    "jobs_in_turn_late": (rand(8, 24, 400, 900), rand(9, 24, 7, 140), 333, 0, 8),
    "long_window": ([6000], [40], 5000, 70, 1),
    "few_queries_many_rows": (rand(10, 300, 9, 60), rand(11, 300, 0, 9), 20, 2, 2),
}


@pytest.mark.parametrize("name", sorted(MANY))
def test_rows_with_several_queries(name):
    seq, qo, window, sinks, Hkv = MANY[name]
    qo = [min(a, b) for a, b in zip(seq, qo)]
    c = Case(seq, qo, window, sinks, Hkv, seed=len(name))
    ws = c.workspace()
    c.check(*c.run(workspace=ws), what=name)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


def test_padding_rows():
    c = Case([300, 0, 40, 0, 0, 1], [1] * 6, 64, 4, 2)
    out, lse = c.decode()
    assert not bool(out[[1, 3, 4]].any()) and bool(torch.isneginf(lse[[1, 3, 4]]).all())
    live = [0, 2, 5]
    d = Case([300, 0, 40, 0, 0, 1], [1, 0, 1, 0, 0, 1], 64, 4, 2)
    d.q, d.d["q"] = c.q[live], c.d["q"][live].contiguous()
    d.k, d.v, d.tables, d.d["k"], d.d["v"], d.d["tables"] = c.k, c.v, c.tables, c.d["k"], c.d["v"], c.d["tables"]
    d.check(out[live], lse[live])


@pytest.mark.parametrize("L", [-1, (1 << 20) + 1, 16 * 19 + 1, -(1 << 31), (1 << 31) - 1])
def test_a_length_out_of_bounds_is_recorded(L):
    c = Case([300, 64, 40], [1] * 3, 64, 4, 2)
    want, _ = c.decode()
    ws = c.workspace()
    c.d["seq"][1] = L
    out, lse = c.decode(workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    assert torch.equal(out[[0, 2]], want[[0, 2]]) and not bool(out[1].any()) and bool(torch.isneginf(lse[1]).all())


@pytest.mark.parametrize("qo", [1, 5, 40])
def test_a_block_outside_the_pool_is_recorded(qo):
    c = Case([200, 90], [qo, qo], 70, 4, 2, seed=3)
    want = c.run()[0]
    c.d["tables"][1, 4] = 10 ** 6
    c.tables[1, 4] = 10 ** 6
    ws = c.workspace()
    out, lse = c.run(workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    assert torch.equal(out[:qo], want[:qo])
    c.check(out, lse)


@pytest.mark.parametrize("qo", [1, 5, 40])
def test_every_key_masked_gives_zero_and_minus_infinity(qo):
    c = Case([40], [qo], 20, 4, 2, seed=5)
    c.d["tables"].fill_(-1)
    out, lse = c.run()
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("scale", [4.0, -0.3, 0.0])
def test_scales(scale):
    c = Case([400, 33, 120], [1, 9, 40], 100, 4, 2, seed=12, scale=scale)
    c.check(*c.run())


def test_without_lse():
    c = Case([400, 33], [1, 9], 100, 4, 2, seed=12)
    d = c.d
    out, _ = c.run()
    alone = B.pa_attention_varlen_window(d["q"], d["k"], d["v"], d["tables"], d["seq"], d["ind"], c.scale, 100, 4)
    assert torch.equal(alone, out)


@pytest.mark.parametrize("qo", [1, 4, 40])
def test_a_query_that_is_not_a_number_shows_and_stays_in_its_row(qo):
    c = Case([300, 90], [qo, qo], 100, 4, 2, seed=6)
    want, want_lse = c.run()
    c.d["q"][0, 3, 7] = float("nan")
    out, lse = c.run()
    keep = torch.ones(2 * qo, 8, dtype=torch.bool, device=DEV)
    keep[0, 3] = False
    assert bool(torch.isnan(out[0, 3]).all()) and bool(torch.isnan(lse[0, 3]))
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


def test_the_same_bits_again():
    c = Case(rand(30, 40, 100, 3000), [1, 3, 9, 50] * 10, 700, 4, 4, seed=7)
    ws = c.workspace()
    out, lse = c.run(workspace=ws)
    for _ in range(5):
        o, l = c.run(workspace=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_rows_behind_the_last_query_are_left():
    c = Case([70, 200], [7, 40], 50, 4, 2, seed=8)
    out = torch.full((60, 8, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    c.check(*c.run(out=out[:47]))
    assert bool((out[47:] == 5.0).all())


def test_a_captured_decode_takes_new_lengths():
    """One captured launch over batches of other lengths, tables and queries,
    its workspace shared with a second graph."""
    R, Hkv, window, sinks = 24, 2, 200, 4
    first = Case([1] * R, [1] * R, window, sinks, Hkv, seed=9)
    nb = 1500
    t = dict(q=torch.zeros(R, 4 * Hkv, 128, dtype=torch.bfloat16, device=DEV), k=torch.zeros(nb, Hkv, 16, 128, dtype=torch.bfloat16, device=DEV),
             tables=torch.full((R, 200), -1, dtype=torch.int32, device=DEV), seq=torch.zeros(R, dtype=torch.int32, device=DEV))
    t["v"] = torch.zeros_like(t["k"])
    ws = first.workspace()
    graphs = []
    for _ in range(2):
        graph, out = torch.cuda.CUDAGraph(), torch.empty_like(t["q"])
        lse = torch.empty(R, 4 * Hkv, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            B.pa_decode_window(t["q"], t["k"], t["v"], t["tables"], t["seq"], first.scale, window, sinks, out=out, lse=lse,
                               workspace=ws)
        graphs.append((graph, out, lse))
    for i in range(6):
        c = Case(rand(40 + i, R, 1, [40, 3000][i % 2]), [1] * R, window, sinks, Hkv, seed=50 + i)
        t["tables"][:, :c.tables.shape[1]].copy_(c.d["tables"])
        for x in ("k", "v"):
            t[x][:c.k.shape[0]].copy_(c.d[x])
        t["q"].copy_(c.d["q"])
        t["seq"].copy_(c.d["seq"])
        graph, out, lse = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse, what=str(i))
    assert B.pa_get_device_error(ws) == 0


def test_on_a_stream_that_is_not_the_current_one():
    c = Case([300, 45, 700], [1, 9, 4], 100, 4, 2, seed=10)
    want, want_lse = c.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = c.run(stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("qo", [1, 2, 5, 8, 40, 130])
@pytest.mark.parametrize("scale", [0.5, -2.0])
def test_scores_that_climb_along_the_keys(qo, scale):
    """Keys that grow along the row, so that every row's reference is raised over and
    over, between tiles without a hidden key too, and by far more than a float's range."""
    c = Case([1800, 700], [qo, qo], 1500, 4, 2, seed=qo, scale=scale)
    x = oracle.bf16_to_f64(c.k)
    for r in range(2):
        for j, b in enumerate(c.tables[r]):
            if b >= 0:
                x[b] *= (1 + j % 40) / 8 * (1 if r else 1 + j / 16)
    k = torch.from_numpy(x).to(torch.bfloat16)
    c.d["k"], c.k = k.to(DEV), bf16_host(k)
    c.check(*c.run())


def test_more_items_than_one_launch_takes():
    R = 1600
    c = Case(rand(20, R, 9, 40), [9] * R, 12, 1, 1, seed=21)
    c.check(*c.run())


@pytest.mark.parametrize("seq,qo,window", [([6000], [100], 5000), ([3000] * 3, [200] * 3, 2500), ([900] * 40, [5] * 40, 700)])
def test_rows_cut_between_processors_give_the_same_bits_again(seq, qo, window):
    c = Case(seq, qo, window, 4, 3, seed=22)
    ws = c.workspace()
    out, lse = c.run(workspace=ws)
    c.check(out, lse)
    for _ in range(8):
        o, l = c.run(workspace=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_threads_with_streams_and_workspaces_of_their_own():
    import threading
    cases = [Case([900, 300, 40], [100, 1, 5], 200, 4, 2, seed=23), Case([2000] * 4, [1, 70, 9, 3], 500, 0, 4, seed=24),
             Case([40] * 30, [1] * 30, 20, 4, 1, seed=25)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            side, ws = torch.cuda.Stream(), cases[i].workspace()
            side.wait_stream(torch.cuda.default_stream())
            for _ in range(30):
                out, lse = cases[i].run(stream=side, workspace=ws)
                side.synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                    wrong.append(i)
        except Exception as e:  # noqa: BLE001 (shown by the assertion)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i % 3,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_a_pool_whose_offsets_pass_32_bits():
    """Blocks at the far end of a pool of more than 2^31 values, written by the append
    and read by each kernel."""
    Hkv, nb = 8, 140_000
    small = Case([600, 350, 90, 33], [70, 1, 5, 1], 200, 4, Hkv, seed=26)
    far = nb - small.k.shape[0]
    k, v = (torch.empty(nb, Hkv, 16, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[far:], v[far:] = small.d["k"], small.d["v"]
    tables = torch.where(small.d["tables"] >= 0, small.d["tables"] + far, small.d["tables"])
    want, want_lse = small.run()
    out, lse = B.pa_attention_varlen_window(small.d["q"], k, v, tables, small.d["seq"], small.d["ind"], small.scale,
                                            small.window, small.sinks, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # the last slot of the pool
    g = torch.Generator(device=DEV).manual_seed(3)
    q, kn, vn = (torch.randn(1, h, 128, generator=g, device=DEV).to(torch.bfloat16) for h in (4 * Hkv, Hkv, Hkv))
    ws = small.workspace()
    slot = torch.tensor([16 * nb - 1], device=DEV)
    turns = B.pa_rope_turns([1.0 / 10000 ** (i / 64) for i in range(64)]).to(DEV)
    before = k[-1, :, :15].clone()
    B.pa_qk_norm_rope_append(q, kn, vn, torch.zeros(1, dtype=torch.int32, device=DEV), slot, turns, k, v, workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    assert torch.equal(k[-1, :, 15], kn[0]) and torch.equal(v[-1, :, 15], vn[0]) and torch.equal(
        k[-1, :, :15].view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("shift", [-3, 1000, (1 << 31) - 40])
def test_a_row_whose_queries_lie_outside_is_recorded_and_left(shift):
    """A device copy of qo_indptr that is not the host's."""
    c = Case([300, 64, 40], [1, 4, 2], 64, 4, 2, seed=31)
    want, want_lse = c.run()
    ws = c.workspace()
    out, lse = torch.full_like(want, 5.0), torch.full_like(want_lse, 5.0)
    wrong = torch.from_numpy(c.ind).clone()
    wrong[2:] += shift                       # (row 1 has another number of queries, row 2 others)
    c.d["ind"].copy_(wrong)
    d = c.d
    B.pa_attention_varlen_window(d["q"], d["k"], d["v"], d["tables"], d["seq"], d["ind"], c.scale, c.window, c.sinks,
                                 seq_lens_host=torch.from_numpy(c.seq), qo_indptr_host=torch.from_numpy(c.ind), out=out,
                                 lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out[:1], want[:1]) and torch.equal(lse[:1], want_lse[:1])
    if shift > 0:
        assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX and bool((out[1:] == 5.0).all())


@pytest.mark.parametrize("most,Hkv,window,sinks", [(1, 3, 100, 4), (1, 8, 300, 17), (1, 2, 1, 1), (2, 2, 150, 0), (3, 8, 20, 0),
                                                   (4, 3, 100, 4)])
def test_many_short_rows(most, Hkv, window, sinks):
    """More rows than segments several times over, some of them empty."""
    R = 500
    rng = np.random.default_rng(most + Hkv)
    seq = rng.integers(1, 141, R)
    qo = np.minimum(rng.integers(0, most + 1, R) if most > 1 else np.ones(R, int), seq)
    qo[7] = min(most, int(seq[7]))
    c = Case(seq.tolist(), qo.tolist(), window, sinks, Hkv, seed=most)
    ws = c.workspace()
    out, lse = c.run(workspace=ws)
    c.check(out, lse)
    again = c.run(workspace=ws) if most > 1 else c.decode(workspace=ws)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    if most == 1:                                # padding rows between (and so other cuts)
        live = np.arange(R) % 3 != 0
        c.d["seq"][torch.from_numpy(~live).to(DEV)] = 0
        out, lse = c.decode(workspace=ws)
        at = torch.from_numpy(live).to(DEV)
        assert not bool(out[~at].any()) and bool(torch.isneginf(lse[~at]).all())
        c.seq, c.qo, c.q = np.where(live, c.seq, 0).astype(np.int32), live.astype(np.int32), c.q[live]
        c.ind = np.concatenate([[0], np.cumsum(c.qo)]).astype(np.int32)
        c.check(out[at], lse[at])
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
