"""q4 KV pages through the C ABI against the oracle: the quantising append and
the read-back are bit-exact, attention over q4 pages is within a bound that is
derived from its own inputs.

Bounds.  Scores: 128 products of bf16 numbers are exact in binary32; summing
them and scaling rounds each at most 2^-24 relative some 136 times, so a score
is off by at most DS = 2^-16 sm_scale max_t sum_d |q_d k_td|.  Then lse is off
by at most DS plus a few roundings of its own, and every probability by a
factor exp(2 DS).  The weights of rows with several queries are rounded to
bf16 (2^-8 each) before the PV product, those of single tokens carry 16 bits;
an output is rounded once to bf16.  With A = sum_t p_t |v_t|:
  |out - ref| <= 2^-8 |ref| + (w + 4 DS + 2^-14) A,  w = 2^-8 or 2^-15.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import q4
from paged_kv_decode_varlen_gb300 import workloads as W
from tests.util import bf16_dev, bf16_host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

DEV = "cuda"


def _pool_pair(nb, Hkv):
    return B.new_q4_pool(nb, Hkv, DEV), B.new_q4_pool(nb, Hkv, DEV)


def _rows(rng, n, Hkv, kind="normal"):
    x = rng.standard_normal((n, Hkv, 128)).astype(np.float32)
    if kind == "offset":      # channels far to one side, of very different sizes
        x = x * np.exp2(rng.integers(-12, 13, (Hkv, 128))).astype(np.float32) + 3 * rng.standard_normal((Hkv, 128))
    elif kind == "constant":
        x = np.repeat(x[..., ::32], 32, -1)
    elif kind == "spread":    # one value of a group far larger than the others
        x[..., ::32] *= 1000
    elif kind == "tiny":
        x = x * np.float32(2.0 ** -130)
    elif kind == "huge":
        x = np.clip(x * np.float32(2.0 ** 125), -2.0 ** 126, 2.0 ** 126)
    return W.f32_to_bf16_bits(x.astype(np.float32))


# ------------------------------------------------------- write and read back
@pytest.mark.parametrize("kind", ["normal", "offset", "constant", "spread", "tiny", "huge"])
@pytest.mark.parametrize("n,Hkv", [(1, 1), (16, 8), (61, 3), (37, 12)])
def test_append_and_read_are_bit_exact(n, Hkv, kind):
    rng = np.random.default_rng(n * 100 + Hkv)
    nb = n // 16 + 3
    k, v = _rows(rng, n, Hkv, kind), _rows(rng, n, Hkv, kind)
    slots = rng.permutation(nb * 16)[:n].astype(np.int64)
    if n > 16:
        slots[5::7] = -1
    kc, vc = _pool_pair(nb, Hkv)
    hk, hv = np.zeros((nb, Hkv, q4.SLAB), np.uint8), np.zeros((nb, Hkv, q4.SLAB), np.uint8)
    q4.append(k, slots, hk)
    q4.append(v, slots, hv)
    st = torch.from_numpy(slots).to(DEV)
    ws = B.pa_kv_append_q4(bf16_dev(k), bf16_dev(v), st, kc, vc)
    ko, vo = B.pa_kv_read_q4(st, kc, vc, workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    assert np.array_equal(kc.cpu().numpy(), hk) and np.array_equal(vc.cpu().numpy(), hv)
    for got, pool in ((ko, hk), (vo, hv)):
        want = q4.unpack(pool)[np.maximum(slots, 0) // 16, :, np.maximum(slots, 0) % 16]
        want[slots < 0] = 0
        assert np.array_equal(bf16_host(got), want)


def test_read_takes_a_slot_many_times_and_records_bad_ones():
    rng = np.random.default_rng(8)
    kc, vc = _pool_pair(4, 2)
    k, v = _rows(rng, 64, 2), _rows(rng, 64, 2)
    ws = B.pa_kv_append_q4(bf16_dev(k), bf16_dev(v), torch.arange(64, device=DEV), kc, vc)
    slots = torch.tensor([3, 3, 63, -5, 64, 3, 1 << 40], device=DEV)
    ko, vo = B.pa_kv_read_q4(slots, kc, vc, workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    assert torch.equal(ko[0], ko[1]) and torch.equal(vo[0], vo[5]) and bool(ko[2].any())
    assert not bool(ko[[3, 4, 6]].any()) and not bool(vo[[3, 4, 6]].any())


def test_append_records_bad_slots_and_leaves_the_rest():
    rng = np.random.default_rng(9)
    kc, vc = _pool_pair(3, 2)
    kc.fill_(0x5a)
    k = _rows(rng, 3, 2)
    ws = B.pa_kv_append_q4(bf16_dev(k), bf16_dev(k), torch.tensor([48, 17, 1 << 50], device=DEV), kc, vc)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    want = np.full((3, 2, q4.SLAB), 0x5a, np.uint8)
    q4.append(k, np.array([-1, 17, -1]), want)
    assert np.array_equal(kc.cpu().numpy(), want)


# ------------------------------------------------------------------ attention
class Case:
    """A batch over q4 pools: cached and new tokens quantised by the oracle,
    every other byte of the pools set to `fill` (0xff: NaN scales)."""

    def __init__(self, seq, qo, Hkv=2, seed=0, fill=0xff, shared=0):
        need = sum(-(-L // 16) for L in seq)
        b = W.make_batch(seq, qo, num_blocks=need + 5, seed=seed, num_q_heads=4 * Hkv, num_kv_heads=Hkv,
                         shared_prefix_tokens=shared)
        self.b, nb = b, need + 5
        self.hk = np.full((nb, Hkv, q4.SLAB), fill, np.uint8)
        self.hv = self.hk.copy()
        rng = np.random.default_rng(seed + 1)
        slots = np.concatenate([b.block_tables[r, np.arange(L) // 16].astype(np.int64) * 16 + np.arange(L) % 16
                                for r, L in enumerate(seq)]) if seq else np.zeros(0, np.int64)
        slots = np.unique(slots)
        kc, vc = torch.from_numpy(self.hk).to(DEV), torch.from_numpy(self.hv).to(DEV)
        k, v = _rows(rng, len(slots), Hkv), _rows(rng, len(slots), Hkv)
        B.pa_kv_append_q4(bf16_dev(k), bf16_dev(v), torch.from_numpy(slots).to(DEV), kc, vc)
        self.kc, self.vc = kc, vc
        self.hk, self.hv = kc.cpu().numpy(), vc.cpu().numpy()
        self.dev = dict(q=bf16_dev(b.q), tables=torch.from_numpy(b.block_tables).to(DEV),
                        seq=torch.from_numpy(b.seq_lens).to(DEV), ind=torch.from_numpy(b.qo_indptr).to(DEV))

    def run(self, **kw):
        d, b = self.dev, self.b
        return B.pa_attention_varlen_q4(d["q"], self.kc, self.vc, d["tables"], d["seq"], d["ind"], b.sm_scale,
                                        seq_lens_host=torch.from_numpy(b.seq_lens),
                                        qo_indptr_host=torch.from_numpy(b.qo_indptr), return_lse=True, **kw)

    def check(self, out, lse, what=""):
        b = self.b
        k, v = q4.unpack(self.hk), q4.unpack(self.hv)
        ref, ref_lse = oracle.attention_varlen(b.q, k, v, b.block_tables, b.seq_lens, b.qo_indptr, b.sm_scale)
        weight, _ = oracle.attention_varlen(b.q, k, v & 0x7fff, b.block_tables, b.seq_lens, b.qo_indptr, b.sm_scale)
        # sum_d |q_d k_d| is at most |q|_1 max|k|, over the tokens of the batch
        finite = oracle.bf16_to_f64(k)
        kmax = np.abs(finite[np.isfinite(finite) & (np.abs(finite) < 1e4)]).max()
        ds = 2.0 ** -16 * b.sm_scale * kmax * np.abs(oracle.bf16_to_f64(b.q)).sum(-1)
        n_q = np.diff(b.qo_indptr)
        w = np.where(np.repeat(n_q, n_q) > 1, 2.0 ** -8, 2.0 ** -15)
        tol = 2.0 ** -8 * np.abs(ref) + (w[:, None] + 4 * ds + 2.0 ** -14)[..., None] * weight
        got = oracle.bf16_to_f64(bf16_host(out))
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5].tolist(),
                               float(np.nanmax(np.abs(got - ref) / tol)))
        lerr = np.abs(lse.cpu().double().numpy() - ref_lse)
        assert np.all(lerr <= ds + 2.0 ** -20 * (1 + np.abs(ref_lse))), (what, float(lerr.max()))


DECODE = {
    "one_token": ([1], 1),
    "page_ends": ([15, 16, 17, 31, 32, 33, 47, 48, 49], 1),
    "three_heads": ([100, 7, 300], 3),
    "twelve_heads": ([129, 64, 1, 500], 12),
    "eight_heads": ([17, 100, 256, 513], 8),
    "long_and_short": ([9000, 1, 40, 2100, 16], 2),
    "many_rows": ([int(x) for x in np.random.default_rng(4).integers(1, 90, 260)], 1),
    "rows_over_one_launch": ([int(x) for x in np.random.default_rng(5).integers(1, 40, 1100)], 1),
}


@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode_rows(name):
    seq, Hkv = DECODE[name]
    c = Case(seq, [1] * len(seq), Hkv, seed=len(seq))
    ws = B.new_workspace(B.pa_attention_workspace_size(len(seq), len(seq), 4 * Hkv, 128, max(seq)), DEV)
    c.check(*c.run(workspace=ws), what=name)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    c.check(*c.run(workspace=ws), what=name + ", the workspace again")


MANY = {
    "whole_prompts": ([1, 16, 17, 33, 129, 250], [1, 16, 17, 33, 129, 250], 2),
    "two_queries": ([2, 300, 17, 16], [2, 2, 2, 2], 3),
    "verify": ([700, 512, 90, 31], [5, 5, 5, 5], 8),
    "chunk_late": ([1500, 600], [70, 33], 1),
    "chunk_tile_edges": ([128, 129, 160, 257, 96], [32, 33, 31, 64, 65], 1),
    "mixed": ([900, 40, 1, 2000, 513, 77], [100, 1, 1, 1, 7, 0], 2),
    "idle_rows": ([50, 0, 30, 70, 9], [0, 0, 3, 0, 1], 2),
    # more jobs than SMs, of one and of two query tiles in every order
    "jobs_in_turn": ([int(x) for x in np.random.default_rng(6).integers(7, 200, 40)],
                     [int(x) for x in np.random.default_rng(7).integers(7, 100, 40)], 8),
    "jobs_in_turn_late": ([int(x) for x in np.random.default_rng(8).integers(400, 900, 24)],
                          [int(x) for x in np.random.default_rng(9).integers(7, 140, 24)], 8),
    "two_to_six_queries": ([40, 2, 333, 16, 17, 90, 3000, 6, 128], [2, 2, 3, 4, 5, 6, 6, 6, 4], 3),
    "few_queries_many_rows": ([int(x) for x in np.random.default_rng(10).integers(6, 60, 300)],
                              [int(x) for x in np.random.default_rng(11).integers(0, 7, 300)], 2),
}


@pytest.mark.parametrize("name", sorted(MANY))
def test_rows_with_several_queries(name):
    seq, qo, Hkv = MANY[name]
    qo = [min(a, b) for a, b in zip(seq, qo)]
    c = Case(seq, qo, Hkv, seed=len(name))
    ws = B.new_workspace(B.pa_attention_workspace_size(len(seq), sum(qo), 4 * Hkv, 128, max(seq)), DEV)
    c.check(*c.run(workspace=ws), what=name)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


@pytest.mark.parametrize("qo", [1, 40])
def test_infinities_in_unused_slots_do_not_leak(qo):
    c = Case([45, 130], [min(qo, 45), qo], 2, seed=qo)
    # D = Z = +-inf in every token slot past the rows' ends
    for r, L in enumerate([45, 130]):
        blk, t = int(c.b.block_tables[r, -1 if r else 2]), L % 16
        for pool, word in ((c.kc, 0x7f80), (c.vc, 0xff80)):
            pool[blk, :, 1024 + 16 * t:] = torch.tensor(np.full(8 * (16 - t), word, np.uint16).view(np.uint8)).to(DEV)
    c.hk, c.hv = c.kc.cpu().numpy(), c.vc.cpu().numpy()
    c.check(*c.run())


@pytest.mark.parametrize("qo", [1, 20])
def test_a_block_outside_the_pool_is_recorded(qo):
    c = Case([200, 90], [qo, qo], 2, seed=3)
    c.dev["tables"][1, 2] = 10 ** 6
    ws = B.new_workspace(B.pa_attention_workspace_size(2, 2 * qo, 8, 128, 200), DEV)
    out, lse = c.run(workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    # the other row is right, and this one is finite
    one = Case([200, 90], [qo, qo], 2, seed=3).run()[0]
    assert torch.equal(out[:qo], one[:qo]) and bool(torch.isfinite(out.float()).all())


def test_every_key_masked_gives_zero_and_minus_infinity():
    c = Case([40], [1], 2, seed=5)
    c.dev["tables"].fill_(-1)
    out, lse = c.run()
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("ctas", [1, 3, 64, 1024])
def test_forced_decode_grid(ctas):
    c = Case([2100, 37, 16, 1, 700, 129], [1] * 6, 2, seed=70 + ctas)
    B.pa_set_decode_ctas(ctas)
    try:
        out, lse = c.run()
        torch.cuda.synchronize()
    finally:
        B.pa_set_decode_ctas(0)
    c.check(out, lse, f"ctas={ctas}")


def test_shared_pages():
    c = Case([700, 900, 650], [1, 4, 1], 2, seed=11, shared=512)
    c.check(*c.run())


def test_large_scores_and_no_lse():
    c = Case([400, 33], [1, 9], 2, seed=12)
    c.b.sm_scale = 4.0     # softmax close to one-hot, scores of some hundreds
    out, lse = c.run()
    c.check(out, lse)
    d = c.dev
    alone = B.pa_attention_varlen_q4(d["q"], c.kc, c.vc, d["tables"], d["seq"], d["ind"], 4.0)
    assert torch.equal(alone, out)


def test_the_pool_may_be_larger_than_four_gigabytes():
    nb = (1 << 32) // (8 * q4.SLAB) + 50
    kc, vc = _pool_pair(nb, 8)
    rng = np.random.default_rng(2)
    L = 70
    k, v = _rows(rng, L, 8), _rows(rng, L, 8)
    blocks = np.array([nb - 1, 0, nb - 2, nb - 40, 1], np.int32)
    slots = blocks[np.arange(L) // 16].astype(np.int64) * 16 + np.arange(L) % 16
    st = torch.from_numpy(slots).to(DEV)
    B.pa_kv_append_q4(bf16_dev(k), bf16_dev(v), st, kc, vc)
    ko, vo = B.pa_kv_read_q4(st, kc, vc)
    small_k, small_v = _pool_pair(5, 8)
    at = torch.arange(L, device=DEV)
    B.pa_kv_append_q4(bf16_dev(k), bf16_dev(v), at, small_k, small_v)
    sk, sv = B.pa_kv_read_q4(at, small_k, small_v)
    assert torch.equal(ko, sk) and torch.equal(vo, sv)
    for qo in (1, 9):
        q = bf16_dev(W.normal_bf16(rng, (qo, 32, 128)))
        args = (torch.tensor([L], dtype=torch.int32, device=DEV), torch.tensor([0, qo], dtype=torch.int32, device=DEV),
                0.088)
        far = B.pa_attention_varlen_q4(q, kc, vc, torch.from_numpy(blocks[None]).to(DEV), *args)
        near = B.pa_attention_varlen_q4(q, small_k, small_v,
                                        torch.arange(5, dtype=torch.int32, device=DEV)[None].contiguous(), *args)
        assert torch.equal(far, near)


# ------------------------------------------------------------ used together
def test_a_serving_sequence_agrees_with_bf16_pages():
    """Prefill in chunks, then decode steps, appending as it goes; the same
    steps over a bf16 pool that holds the rows read back."""
    rng = np.random.default_rng(21)
    Hkv, blocks = 2, 40
    kc, vc = _pool_pair(blocks, Hkv)
    kb = torch.zeros(blocks, Hkv, 16, 128, dtype=torch.bfloat16, device=DEV)
    vb = torch.zeros_like(kb)
    tables = torch.from_numpy(rng.permutation(blocks)[:36].reshape(2, 18).astype(np.int32)).to(DEV)
    ws = B.new_workspace(B.pa_attention_workspace_size(2, 200, 4 * Hkv, 128, 288), DEV)
    lens = [0, 0]
    for new in ([100, 37], [90, 1], [1, 1], [1, 0], [1, 1], [0, 5]):
        lens = [a + n for a, n in zip(lens, new)]
        total = sum(new)
        slots = torch.cat([tables[r, torch.arange(L - n, L, device=DEV) // 16].long() * 16 +
                           torch.arange(L - n, L, device=DEV) % 16 for r, (L, n) in enumerate(zip(lens, new))])
        k, v = bf16_dev(_rows(rng, total, Hkv)), bf16_dev(_rows(rng, total, Hkv))
        B.pa_kv_append_q4(k, v, slots, kc, vc, workspace=ws)
        ko, vo = B.pa_kv_read_q4(slots, kc, vc, workspace=ws)
        B.pa_kv_append(ko, vo, slots, kb, vb, workspace=ws)
        q = bf16_dev(W.normal_bf16(rng, (total, 4 * Hkv, 128)))
        seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
        ind = torch.tensor([0, new[0], total], dtype=torch.int32, device=DEV)
        out, lse = B.pa_attention_varlen_q4(q, kc, vc, tables, seq, ind, 0.088, return_lse=True, workspace=ws)
        ref, ref_lse = B.pa_attention_varlen(q, kb, vb, tables, seq, ind, 0.088, return_lse=True, workspace=ws)
        # both within 2^-8 |ref| + (2^-8 + ..) A of the same definition; A <= max |v| ~ 4.5
        assert float((out.float() - ref.float()).abs().max()) <= 2 * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -12) * 4.5
        assert float((lse - ref_lse).abs().max()) <= 1e-4
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


def test_captured_step_replays_on_new_contents_and_other_streams():
    c = Case([300, 45, 700, 64], [1, 1, 6, 1], 2, seed=31)
    d, b = c.dev, c.b
    total = int(b.qo_indptr[-1])
    k, v = bf16_dev(b.k_new), bf16_dev(b.v_new)
    slots = torch.from_numpy(b.slot_mapping).to(DEV)
    ws = B.new_workspace(B.pa_attention_workspace_size(4, total, 8, 128, 700), DEV)
    out = torch.empty_like(d["q"])
    lse = torch.empty(total, 8, dtype=torch.float32, device=DEV)

    def step():
        B.pa_kv_append_q4(k, v, slots, c.kc, c.vc, workspace=ws)
        c.run(out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = np.random.default_rng(32)
    for _ in range(2):
        k.copy_(bf16_dev(_rows(rng, total, 2)))
        v.copy_(bf16_dev(_rows(rng, total, 2)))
        b.q[:] = W.normal_bf16(rng, b.q.shape)
        d["q"].copy_(bf16_dev(b.q))
        g.replay()
        torch.cuda.synchronize()
        c.hk, c.hv = c.kc.cpu().numpy(), c.vc.cpu().numpy()
        c.check(out, lse)
    assert B.pa_get_device_error(ws) == 0


def test_calls_on_two_streams_with_workspaces_of_their_own():
    cases = [Case([1200, 300], [1, 1], 2, seed=41), Case([900, 64, 77], [1, 30, 1], 2, seed=42)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append([c.run() for _ in range(5)])
    torch.cuda.synchronize()
    for c, runs in zip(cases, got):
        for out, lse in runs:
            c.check(out, lse)
            assert torch.equal(out, runs[0][0])


# --------------------------------------------- calls that a rule sends elsewhere
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, -1e-44])
def test_zero_negative_and_tiny_scales(scale):
    c = Case([300, 33, 150, 70], [1, 4, 90, 40], 2, seed=51)
    c.b.sm_scale = scale
    out, lse = c.run()
    c.b.sm_scale = abs(scale)
    if scale < 0:  # for the oracle the sign goes to q
        c.b.q[:] ^= np.uint16(0x8000)
    c.check(out, lse, f"scale {scale}")


@pytest.mark.parametrize("qo,scale", [(1, 1e36), (2, 1e36), (6, 1e36), (7, 1e6), (40, 1e6)])
def test_very_large_scores(qo, scale):
    """A row's first query of a whole prompt sees one key: the output is its
    value (to the rounding of the weight and of the output, 2^-8 each), lse its
    score."""
    c = Case([qo, qo], [qo, qo], 2, seed=52)
    c.b.sm_scale = scale
    out, lse = c.run()
    k, v, q = (oracle.bf16_to_f64(x) for x in (q4.unpack(c.hk), q4.unpack(c.hv), c.b.q))
    got = oracle.bf16_to_f64(bf16_host(out))
    for r in range(2):
        blk = int(c.b.block_tables[r, 0])
        for h in range(8):
            key, val = k[blk, h // 4, 0], v[blk, h // 4, 0]
            assert np.all(np.abs(got[r * qo, h] - val) <= 2.0 ** -7 * np.abs(val) * (1 + 2.0 ** -6))
            score = scale * float(q[r * qo, h] @ key)
            # 128 products and sums in binary32, then the scale's roundings
            assert abs(float(lse[r * qo, h]) - score) <= 2.0 ** -16 * scale * float(np.abs(q[r * qo, h]) @ np.abs(key))
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("qo", [[1, 1], [5, 5], [90, 40]])
def test_views_at_sixteen_byte_offsets(qo):
    c = Case([200, 61], qo if qo[1] <= 61 else [90, 40], 2, seed=54)
    want, want_lse = c.run()
    d, total = c.dev, int(c.b.qo_indptr[-1])

    def shifted(t, fill=0):
        buf = torch.full((t.numel() + 8,), fill, dtype=t.dtype, device=DEV)
        view = buf[8:].view(t.shape)  # 16 bytes of bf16
        return buf, view

    _, q = shifted(d["q"])
    q.copy_(d["q"])
    obuf, out = shifted(want, 7)
    pools = []
    for pool in (c.kc, c.vc):
        buf = torch.empty(pool.numel() + 16, dtype=torch.uint8, device=DEV)
        pools.append(buf[16:].view(pool.shape))
        pools[-1].copy_(pool)
    got, lse = B.pa_attention_varlen_q4(q, pools[0], pools[1], d["tables"], d["seq"], d["ind"], c.b.sm_scale, out=out,
                                        return_lse=True)
    assert torch.equal(got, want) and torch.equal(lse, want_lse) and got.shape[0] == total
    assert bool((obuf[:8] == 7).all())


def test_tile_jobs_beside_the_decode_launch_or_before_it():
    c = Case([1500, 1200, 900, 800, 300, 700], [100, 1, 1, 1, 1, 1], 2, seed=55)
    out, lse = c.run()
    c.check(out, lse, "as planned")
    B.pa_set_prefill_ctas(-1)
    try:
        first, first_lse = c.run()
        torch.cuda.synchronize()
    finally:
        B.pa_set_prefill_ctas(0)
    c.check(first, first_lse, "one after the other")
    assert torch.equal(first[:100], out[:100])  # the tile jobs' own rows do not depend on it


def test_results_do_not_depend_on_what_the_workspace_held():
    sizes = [([900, 1500], [1, 1]), ([300] * 70, [1] * 70), ([4000], [5]), ([64, 2000, 31], [64, 1, 3])]
    cases = [Case(s, q, 2, seed=56 + i) for i, (s, q) in enumerate(sizes)]
    need = max(B.pa_attention_workspace_size(len(s), sum(q), 8, 128, max(s)) for s, q in sizes)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device=DEV)
    ws[:B.PA_ERROR_WORD_BYTES] = 0
    clean = [c.run() for c in cases]
    for _ in range(2):
        for c, (out, lse) in zip(cases, clean):
            got, got_lse = c.run(workspace=ws)
            assert torch.equal(got, out) and torch.equal(got_lse, lse)
    ws[B.PA_ERROR_WORD_BYTES:] = 0xff
    for c, (out, _) in zip(reversed(cases), reversed(clean)):
        assert torch.equal(c.run(workspace=ws)[0], out)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


def test_two_graphs_share_a_workspace():
    cases = [Case([2500, 40], [1, 1], 2, seed=61), Case([700, 650, 90], [3, 1, 20], 2, seed=62)]
    ws = B.new_workspace(max(B.pa_attention_workspace_size(len(c.b.seq_lens), int(c.b.qo_indptr[-1]), 8, 128, 2500)
                             for c in cases), DEV)
    want = [c.run() for c in cases]
    outs, graphs = [], []
    for c in cases:
        out, lse = torch.empty_like(c.dev["q"]), torch.empty(c.dev["q"].shape[:2], device=DEV)
        c.run(out=out, lse=lse, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=out, lse=lse, workspace=ws)
        outs.append((out, lse))
        graphs.append(g)
    for order in ([0, 1], [1, 0, 0, 1, 1]):
        for out, lse in outs:
            out.zero_()
            lse.zero_()
        for i in order:
            graphs[i].replay()
        for (out, lse), (w, wl) in zip(outs, want):
            assert torch.equal(out, w) and torch.equal(lse, wl)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


def test_rows_behind_the_last_sequence_stay():
    c = Case([77, 130, 20], [1, 40, 3], 2, seed=63)
    want, want_lse = c.run()
    total = want.shape[0]
    big = torch.full((total + 90, 8, 128), -5.0, dtype=torch.bfloat16, device=DEV)
    biglse = torch.full((total + 90, 8), -5.0, device=DEV)
    c.run(out=big[:total], lse=biglse[:total])
    assert torch.equal(big[:total], want) and torch.equal(biglse[:total], want_lse)
    assert bool((big[total:] == -5).all()) and bool((biglse[total:] == -5).all())
    kc, vc = _pool_pair(4, 2)
    k = bf16_dev(_rows(np.random.default_rng(64), 9, 2))
    B.pa_kv_append_q4(k, k, torch.arange(9, device=DEV), kc, vc)
    buf = torch.full((15, 2, 128), -5.0, dtype=torch.bfloat16, device=DEV)
    B.pa_kv_read_q4(torch.arange(9, device=DEV), kc, vc, k_out=buf[:9], v_out=torch.empty_like(k))
    assert bool((buf[9:] == -5).all()) and not bool((buf[:9] == -5).all())


@pytest.mark.parametrize("qo", [1, 6])
def test_rows_of_a_million_pages(qo):
    """A table that names eight blocks over and over: every key counts as often
    as its block is named, so the output is that of the eight blocks and lse is
    greater by the logarithm of their number."""
    Hkv, times = 256, 1100  # 8800 pages x 256 heads: no decode plan
    c = Case([128], [qo], Hkv, seed=65)
    out, lse = c.run()
    q = c.dev["q"]
    tables = c.dev["tables"][:, :8].repeat(1, times).contiguous()
    L = 128 * times
    seq = torch.tensor([L], dtype=torch.int32, device=DEV)
    ind = torch.tensor([0, qo], dtype=torch.int32, device=DEV)
    got, got_lse = B.pa_attention_varlen_q4(q, c.kc, c.vc, tables, seq, ind, c.b.sm_scale, return_lse=True)
    # the last query sees every key.  Each output is off by at most its weights'
    # rounding (2^-8 of max |v|) and half of its own (2^-8): twice that, and the
    # sums of 140800 weights in binary32, in steps of 64 (2^-24 each)
    a, b = got[-1].double(), out[-1].double()
    v = oracle.bf16_to_f64(q4.unpack(c.hv))[c.b.block_tables[0, :8]]
    big = float(np.abs(v).max())
    assert float((a - b).abs().max()) <= (4 * 2.0 ** -8 + 2.0 ** -12) * big
    assert float((got_lse[-1] - lse[-1] - np.log(times)).abs().max()) <= 2.0 ** -12


# few tile jobs and many keys: the keys are cut into ranges
RANGES = {
    "one_chunk": ([3000], [20], 2),
    "two_tiles": ([5000, 700], [64, 9], 1),
    "many_ranges": ([20000], [7], 8),
    "ends_inside_a_page": ([4097, 2049], [33, 10], 3),
    "a_whole_prompt": ([600], [600], 1),
    "ranges_that_early_queries_do_not_see": ([260, 1030], [200, 130], 1),
    "beside_decode_rows": ([9000, 900, 30, 2000], [40, 1, 1, 1], 2),
    "beside_verify_rows": ([6000, 900, 30, 0, 2000], [12, 5, 5, 0, 5], 4),
    "before_two_kinds_of_rows": ([7000, 900, 30], [70, 5, 1], 2),
}


@pytest.mark.parametrize("name", sorted(RANGES))
def test_few_jobs_over_many_keys(name):
    seq, qo, Hkv = RANGES[name]
    c = Case(seq, qo, Hkv, seed=70 + len(name))
    need = B.pa_attention_workspace_size(len(seq), sum(qo), 4 * Hkv, 128, max(seq))
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)  # and nothing behind what was asked for
    ws[:B.PA_ERROR_WORD_BYTES] = 0
    B.pa_trace_enable(True)
    try:
        out, lse = c.run(workspace=ws)
        kinds = [k for k, _ in B.pa_trace_read()]
    finally:
        B.pa_trace_enable(False)
    c.check(out, lse, what=name)
    assert kinds.count("prefill") == 1 and kinds.count("merge") == 1, kinds
    again, again_lse = c.run(workspace=ws)
    assert torch.equal(again, out) and torch.equal(again_lse, lse)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0 and bool((ws[need:] == 0xff).all())


def test_ranges_with_a_page_outside_the_pool_and_hidden_ones():
    c = Case([3000], [20], 2, seed=90)
    c.dev["tables"][0, 5] = -7
    ws = B.new_workspace(B.pa_attention_workspace_size(1, 20, 8, 128, 3000), DEV)
    out, lse = c.run(workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    c.dev["tables"].fill_(10 ** 8)
    out, lse = c.run()
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())


def test_captured_key_ranges_replay_beside_other_work():
    c = Case([3000, 500, 40], [20, 1, 1], 2, seed=91)
    want, want_lse = c.run()
    ws = B.new_workspace(B.pa_attention_workspace_size(3, 22, 8, 128, 3000), DEV)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    c.run(out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, lse=lse, workspace=ws)
    other = Case([1200] * 3, [1, 30, 4], 2, seed=92)
    other_want = other.run()[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out.zero_()
        g.replay()
        with torch.cuda.stream(side):
            other_out = other.run(stream=side)[0]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(other_out, other_want)
    assert B.pa_get_device_error(ws) == 0
