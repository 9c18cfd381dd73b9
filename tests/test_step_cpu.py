"""Step tables, norms and rotations, and attention with a window, without a
GPU: their oracles against what fixes them, and the refusals of the calls (no
call here reaches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import step
from paged_kv_decode_varlen_gb300 import binding as b
from paged_kv_decode_varlen_gb300 import workloads as W

lib = b._lib
FAKE = ctypes.c_void_p(1 << 20)  # non-null, aligned; never dereferenced on these paths
ODD = ctypes.c_void_p((1 << 20) + 2)


# ------------------------------------------------------------------- oracles
def test_tables_of_a_small_step():
    # three requests: 15 tokens and one more, a prompt of 20, one that waits
    tables = np.full((3, 4), -1, np.int32)
    tables[0, 0], tables[2, :2] = 7, (1, 2)
    ring = np.array([3, 5, -1, -1, -1, -1, -1, 4], np.int32)
    got, errors = step.step_tables([1, 20, 0], [15, 0, 30], [0, 0, 0], tables, ring, [7, 3], 0, 0, 0, 23)
    assert not errors
    assert got["seq_lens"].tolist() == [16, 20, 30] and got["qo_indptr"].tolist() == [0, 1, 21, 21]
    assert got["block_tables"].tolist() == [[7, -1, -1, -1], [4, 3, -1, -1], [1, 2, -1, -1]]
    assert got["slot_mapping"].tolist() == [7 * 16 + 15] + list(range(64, 80)) + list(range(48, 52)) + [-1, -1]
    assert got["positions"].tolist() == [15] + list(range(20)) + [0, 0]
    assert got["free_state"].tolist() == [1, 1]


def test_tables_give_back_what_no_query_sees():
    # window 20, one sink page: the query at 52 sees 33 .. 52, so page 1 (16 .. 31) goes
    tables = np.array([[0, 1, 2, 3, -1]], np.int32)
    ring = np.array([9, 8, 7, 6, 5, 4, 0, 0, 0, 0], np.int32)
    got, _ = step.step_tables([1], [52], [0], tables, ring, [0, 6], 20, 3, 0, 1)
    assert got["free_state"].tolist() == [0, 7] and got["free_ring"][6] == 1 and got["first_page"].tolist() == [2]
    got, _ = step.step_tables([1], [51], [2], tables, ring, [0, 6], 20, 3, 0, 1)     # already gone
    assert got["free_state"].tolist() == [0, 6] and got["first_page"].tolist() == [2]
    got, _ = step.step_tables([-1], [52], [2], tables, ring, [0, 6], 20, 3, 0, 0)    # the end: pages 0, 2, 3
    assert got["free_ring"][6:9].tolist() == [0, 2, 3] and got["seq_lens"].tolist() == [0]
    got, _ = step.step_tables([-1], [52], [0], tables, ring, [0, 6], 0, 3, 1, 0)     # page 0 is shared
    assert got["free_ring"][6:9].tolist() == [1, 2, 3]


def test_rotation_turns_pairs_and_keeps_their_length():
    rng = np.random.default_rng(2)
    x = W.normal_bf16(rng, (5, 2, 128))
    f = 1e4 ** (-np.arange(32) / 32)
    for inter in (False, True):
        y, _ = step.norm_rope(x, None, np.array([0, 1, 7, 1000, 10 ** 6]), f, 0.0, inter)
        v = oracle.bf16_to_f64(x)
        assert np.array_equal(y[0], v[0]) and np.array_equal(y[:, :, 64:], v[:, :, 64:])
        ia, ib = (np.arange(0, 64, 2), np.arange(1, 64, 2)) if inter else (np.arange(32), np.arange(32, 64))
        assert np.allclose(np.hypot(y[..., ia], y[..., ib]), np.hypot(v[..., ia], v[..., ib]), rtol=1e-12)
        # position 1 at speed 1 turns the first pair by one radian
        a = np.arctan2(y[1, :, ib[0]], y[1, :, ia[0]]) - np.arctan2(v[1, :, ib[0]], v[1, :, ia[0]])
        assert np.allclose((a + np.pi) % (2 * np.pi) - np.pi, 1.0, atol=1e-12)


def test_scores_of_rotated_rows_depend_on_the_distance_alone():
    rng = np.random.default_rng(3)
    x = W.normal_bf16(rng, (2, 1, 128))
    f = 1e6 ** (-np.arange(64) / 64)
    dots = []
    for p in (0, 5, 4321):
        y, _ = step.norm_rope(x, np.ones(128, np.float32), np.array([p, p + 9]), f, 1e-6, False)
        dots.append((y[0, 0] * y[1, 0]).sum())
    assert np.allclose(dots, dots[0], rtol=1e-9)


def test_a_wide_window_is_plain_attention():
    bt = W.make_batch([40, 70, 5], [3, 1, 0], num_blocks=12, seed=4, num_q_heads=8, num_kv_heads=2)
    ref, ref_lse = oracle.attention_varlen(bt.q, bt.k_cache, bt.v_cache, bt.block_tables, bt.seq_lens, bt.qo_indptr,
                                           bt.sm_scale)
    for window, sinks in ((70, 0), (10 ** 6, 5), (1, 70)):
        out, lse, _ = step.attention_window(bt.q, bt.k_cache, bt.v_cache, bt.block_tables, bt.seq_lens, bt.qo_indptr,
                                            bt.sm_scale, window, sinks)
        assert np.allclose(out, ref, atol=1e-9) and np.allclose(lse, ref_lse, atol=1e-9)


def test_a_window_of_one_gives_the_own_value_and_sinks_their_share():
    bt = W.make_batch([40], [2], num_blocks=4, seed=5, num_q_heads=4, num_kv_heads=1)
    zero = np.zeros_like(bt.q)
    out, lse, _ = step.attention_window(zero, bt.k_cache, bt.v_cache, bt.block_tables, bt.seq_lens, bt.qo_indptr, 1.0, 1, 0)
    v = oracle.bf16_to_f64(bt.v_cache)
    own = v[bt.block_tables[0, 2], 0, 6:8]
    assert np.allclose(out[:, 0], own) and np.allclose(lse, 0)
    out, lse, _ = step.attention_window(zero, bt.k_cache, bt.v_cache, bt.block_tables, bt.seq_lens, bt.qo_indptr, 1.0, 1, 3)
    assert np.allclose(out[:, 0], (own + v[bt.block_tables[0, 0], 0, :3].sum(0)) / 4) and np.allclose(lse, np.log(4))


# --------------------------------------------------------------------- turns
def test_turns_are_the_fractions_of_a_turn():
    f = [0.0, 1.0, 2 * np.pi, 0.5 * np.pi, -0.5 * np.pi, 1e-12, 1e9]
    got = b.pa_rope_turns(f).numpy().view(np.uint64)
    want = [(x / (2 * np.pi)) % 1.0 for x in f]
    # a double's relative error 2^-53 in the quotient and in 2 pi, of whole turns too
    for g, w, x in zip(got, want, f):
        d = abs(float(g) * 2.0 ** -64 - w)
        assert min(d, 1 - d) <= 2.0 ** -51 * max(1.0, abs(x)), (g, w)
    assert got[0] == 0 and got[3] == 1 << 62 and got[4] == 3 << 62
    assert b.pa_rope_turns([]).shape == (0,)
    assert b.pa_rope_turns(torch.ones(64)).shape == (64,)


@pytest.mark.parametrize("f", [[float("nan")], [float("inf")], [1.0] * 65])
def test_turns_refuse(f):
    with pytest.raises(b.PAError) as e:
        b.pa_rope_turns(f)
    assert e.value.status == b.PA_ERR_INVALID_ARG


# ------------------------------------------------------------------ refusals
def _tables(**kw):
    a = dict(new=FAKE, cached=FAKE, first=None, R=4, bt=FAKE, mb=8, ring=FAKE, nb=64, state=FAKE, window=0, sinks=0,
             shared=0, n=4, seq=FAKE, ind=FAKE, slots=FAKE, pos=FAKE, so=FAKE, fo=None, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.pa_step_tables(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), b.PA_ERR_INVALID_ARG), (dict(R=65536), b.PA_ERR_INVALID_ARG), (dict(n=-1), b.PA_ERR_INVALID_ARG),
    (dict(nb=0), b.PA_ERR_INVALID_ARG), (dict(nb=1 << 31), b.PA_ERR_INVALID_ARG), (dict(mb=0), b.PA_ERR_INVALID_ARG),
    (dict(window=-1), b.PA_ERR_INVALID_ARG), (dict(sinks=-1), b.PA_ERR_INVALID_ARG),
    (dict(shared=-1), b.PA_ERR_INVALID_ARG), (dict(window=4), b.PA_ERR_INVALID_ARG),        # no first_page_out
    (dict(first=FAKE), b.PA_ERR_INVALID_ARG), (dict(wsb=255), b.PA_ERR_WORKSPACE_TOO_SMALL),
    (dict(ws=ctypes.c_void_p((1 << 20) + 16)), b.PA_ERR_INVALID_ARG), (dict(slots=ctypes.c_void_p((1 << 20) + 4)), b.PA_ERR_INVALID_ARG),
] + [({k: None}, b.PA_ERR_INVALID_ARG) for k in ("new", "cached", "bt", "ring", "state", "seq", "ind", "slots", "pos", "so", "ws")]
  + [({k: ODD}, b.PA_ERR_INVALID_ARG) for k in ("new", "cached", "bt", "ring", "state", "seq", "ind", "pos", "so")])
def test_step_tables_refuses(kw, status):
    assert _tables(**kw) == status
    assert lib.pa_last_error_message().decode()


def _rope(**kw):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, pos=FAKE, n=4, qw=FAKE, kw=None, eps=1e-6, turns=FAKE, rot=128, inter=0,
             Hq=32, Hkv=8, D=128, qo=FAKE, ko=FAKE)
    a.update(kw)
    return lib.pa_qk_norm_rope(*a.values(), None)


def _append(**kw):
    a = dict(q=FAKE, qs=6144, k=FAKE, ks=6144, v=FAKE, vs=6144, pos=FAKE, slots=FAKE, n=4, qw=None, kw=FAKE, eps=0.0,
             turns=FAKE, rot=64, inter=1, Hq=32, Hkv=8, D=128, P=16, qo=FAKE, kc=FAKE, vc=FAKE, nb=4, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.pa_qk_norm_rope_append(*a.values(), None)


BOTH = [(dict(n=-1), b.PA_ERR_INVALID_ARG), (dict(n=1 << 31), b.PA_ERR_UNSUPPORTED), (dict(qs=4088), b.PA_ERR_INVALID_ARG),
        (dict(qs=4100), b.PA_ERR_INVALID_ARG), (dict(ks=1016), b.PA_ERR_INVALID_ARG), (dict(rot=8), b.PA_ERR_INVALID_ARG),
        (dict(rot=-16), b.PA_ERR_INVALID_ARG), (dict(rot=144), b.PA_ERR_INVALID_ARG), (dict(inter=2), b.PA_ERR_INVALID_ARG),
        (dict(eps=-1.0), b.PA_ERR_INVALID_ARG), (dict(eps=float("nan")), b.PA_ERR_INVALID_ARG),
        (dict(eps=float("inf")), b.PA_ERR_INVALID_ARG), (dict(Hq=16), b.PA_ERR_UNSUPPORTED),
        (dict(D=64), b.PA_ERR_UNSUPPORTED), (dict(Hkv=0), b.PA_ERR_INVALID_ARG)] \
    + [({k: None}, b.PA_ERR_INVALID_ARG) for k in ("q", "k", "pos", "turns", "qo")] \
    + [({k: ODD}, b.PA_ERR_INVALID_ARG) for k in ("q", "k", "pos", "turns", "qo", "qw", "kw")]


@pytest.mark.parametrize("kw,status", BOTH + [(dict(ko=None), b.PA_ERR_INVALID_ARG), (dict(ko=ODD), b.PA_ERR_INVALID_ARG)])
def test_norm_rope_refuses(kw, status):
    assert _rope(**kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(vs=1000), b.PA_ERR_INVALID_ARG), (dict(vs=6148), b.PA_ERR_INVALID_ARG), (dict(nb=0), b.PA_ERR_INVALID_ARG),
    (dict(P=32), b.PA_ERR_UNSUPPORTED), (dict(wsb=128), b.PA_ERR_WORKSPACE_TOO_SMALL)]
    + [({k: None}, b.PA_ERR_INVALID_ARG) for k in ("v", "slots", "kc", "vc", "ws")]
    + [({k: ODD}, b.PA_ERR_INVALID_ARG) for k in ("v", "slots", "kc", "vc", "ws")])
def test_norm_rope_append_refuses(kw, status):
    assert _append(**kw) == status


def test_no_tokens_launch_nothing():
    before = b.pa_launch_count()
    assert _rope(n=0, q=None, k=None, pos=None, qo=None, ko=None) == b.PA_OK
    assert _append(n=0, q=None, k=None, v=None, slots=None, pos=None, qo=None) == b.PA_OK
    assert b.pa_launch_count() == before


def _attn(seq=(17, 100), ind=(0, 1, 2), **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, nb=64, bt=FAKE, mb=40, sl=FAKE, qi=FAKE, slh=(ctypes.c_int32 * 2)(*seq),
             qih=(ctypes.c_int32 * 3)(*ind), R=2, tq=2, Hq=32, Hkv=8, D=128, P=16, scale=0.088, window=64, sinks=4,
             out=FAKE, lse=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.pa_attention_varlen_window(*a.values(), None)


def _decode(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, nb=64, bt=FAKE, mb=40, sl=FAKE, R=2, Hq=32, Hkv=8, D=128, P=16, scale=0.088, window=64,
             sinks=4, out=FAKE, lse=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.pa_decode_window(*a.values(), None)


WINDOW = [(dict(D=64), b.PA_ERR_UNSUPPORTED), (dict(P=32), b.PA_ERR_UNSUPPORTED), (dict(Hq=16), b.PA_ERR_UNSUPPORTED),
          (dict(Hkv=0), b.PA_ERR_INVALID_ARG), (dict(nb=0), b.PA_ERR_INVALID_ARG), (dict(scale=float("inf")), b.PA_ERR_INVALID_ARG),
          (dict(scale=float("nan")), b.PA_ERR_INVALID_ARG), (dict(window=0), b.PA_ERR_INVALID_ARG),
          (dict(window=-5), b.PA_ERR_INVALID_ARG), (dict(sinks=-1), b.PA_ERR_INVALID_ARG), (dict(R=-1), b.PA_ERR_INVALID_ARG),
          (dict(R=65536), b.PA_ERR_INVALID_ARG), (dict(wsb=255), b.PA_ERR_WORKSPACE_TOO_SMALL),
          (dict(ws=ctypes.c_void_p((1 << 20) + 16)), b.PA_ERR_INVALID_ARG)] \
    + [({k: None}, b.PA_ERR_INVALID_ARG) for k in ("q", "k", "v", "bt", "sl", "out", "ws")] \
    + [({k: ODD}, b.PA_ERR_INVALID_ARG) for k in ("q", "k", "v", "bt", "sl", "out", "lse", "ws")]


@pytest.mark.parametrize("kw,status", WINDOW + [
    (dict(ind=(0, 1, 3)), b.PA_ERR_INVALID_ARG), (dict(ind=(1, 1, 2)), b.PA_ERR_INVALID_ARG),
    (dict(ind=(0, 2, 1), tq=1), b.PA_ERR_INVALID_ARG), (dict(seq=(0, 100)), b.PA_ERR_INVALID_ARG),
    (dict(seq=(17, 1000)), b.PA_ERR_INVALID_ARG), (dict(seq=(17, (1 << 20) + 1)), b.PA_ERR_UNSUPPORTED),
    (dict(seq=(17, -1)), b.PA_ERR_INVALID_ARG), (dict(slh=None), b.PA_ERR_INVALID_ARG), (dict(qih=None), b.PA_ERR_INVALID_ARG),
    (dict(qi=None), b.PA_ERR_INVALID_ARG), (dict(tq=-1), b.PA_ERR_INVALID_ARG)])
def test_attention_with_a_window_refuses(kw, status):
    if kw.get("R", 2) > 2:  # refused before the host arrays are read
        assert _attn(**kw) == status
        return
    assert _attn(**kw) == status
    assert lib.pa_last_error_message().decode()


@pytest.mark.parametrize("kw,status", WINDOW + [(dict(mb=0), b.PA_ERR_INVALID_ARG)])
def test_decode_with_a_window_refuses(kw, status):
    assert _decode(**kw) == status


def test_empty_batches_launch_nothing():
    before = b.pa_launch_count()
    assert _attn(seq=(5, 0), ind=(0, 0, 0), tq=0, q=None, out=None) == b.PA_OK
    assert _decode(R=0, q=None, out=None, bt=None, sl=None) == b.PA_OK
    assert b.pa_launch_count() == before


def test_window_workspace_query():
    assert b.pa_window_workspace_size(-1, 1, 32, 128, 64, 0) == 0
    small = b.pa_window_workspace_size(1, 1, 32, 128, 64, 0)
    big = b.pa_window_workspace_size(64, 2048, 32, 128, 1 << 30, 1 << 30)
    assert b.PA_ERROR_WORD_BYTES <= small <= big and small % 256 == 0 and big % 256 == 0


# ------------------------------------------------------- the binding's checks
def test_binding_refuses_host_tensors_and_odd_shapes():
    q, k = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    pos, turns = torch.zeros(3, dtype=torch.int32), torch.zeros(64, dtype=torch.int64)
    pool, table = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.int32)
    if torch.cuda.is_available():
        pytest.skip("host tensors are refused by the same check there; a device index is needed for it here")
    b_dev, b._current_device = b._current_device, lambda: 0
    try:
        for call in (lambda: b.pa_qk_norm_rope(q, k, pos, turns, q_out=q, k_out=k),
                     lambda: b.pa_qk_norm_rope(q, k, pos[:2], turns, q_out=q, k_out=k),
                     lambda: b.pa_qk_norm_rope(q, k, pos, turns, q_out=q[:2], k_out=k),
                     lambda: b.pa_decode_window(q, pool, pool, table, pos, 1.0, 8, out=q, workspace=pos),
                     lambda: b.pa_decode_window(q, pool, pool, table[:2], pos, 1.0, 8, out=q, workspace=pos),
                     lambda: b.pa_step_tables(pos, pos, table, pos, pos[:2], n_tokens=3, seq_lens=pos[:2], qo_indptr=pos,
                                              slot_mapping=turns[:3], positions=pos, free_state_out=pos[:2],
                                              first_page_out=pos, workspace=pos)):
            with pytest.raises(ValueError):
                call()
        with pytest.raises(TypeError):
            b.pa_qk_norm_rope(q, k, pos.long(), turns, q_out=q, k_out=k)
    finally:
        b._current_device = b_dev
