"""A decode layer without the host: pa_step_tables, pa_qk_norm_rope_append and
pa_decode_window captured in one graph and replayed step by step, against the
oracles of the three walked the same way."""
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


@pytest.mark.parametrize("Hkv,window,sinks", [(2, 40, 4), (8, 16, 0)])
def test_a_captured_layer_over_many_steps(Hkv, window, sinks):
    """Requests grow from nothing; pages behind their windows come back and are
    granted again, so what was cached is overwritten while others still read."""
    R, nb, max_blocks, steps = 5, 28, 40, 160
    rng = np.random.default_rng(Hkv)
    scale = float(np.float32(128 ** -0.5))
    f = 1e4 ** (-np.arange(64) / 64)
    qw, kw = ((1 + 0.2 * rng.standard_normal(128)).astype(np.float32) for _ in range(2))
    i32 = dict(dtype=torch.int32, device=DEV)
    new, lens, first = torch.ones(R, **i32), torch.zeros(R, **i32), torch.zeros(R, **i32)
    tables, ring, state = torch.full((R, max_blocks), -1, **i32), torch.arange(nb, **i32), torch.tensor([0, nb], **i32)
    ind, slots, pos = torch.zeros(R + 1, **i32), torch.zeros(R, dtype=torch.int64, device=DEV), torch.zeros(R, **i32)
    qkv = torch.zeros(R, 6 * Hkv, 128, dtype=torch.bfloat16, device=DEV)
    q_out, out = (torch.zeros(R, 4 * Hkv, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lse = torch.zeros(R, 4 * Hkv, device=DEV)
    kc = torch.full((nb, Hkv, 16, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    turns, dqw, dkw = B.pa_rope_turns(f).to(DEV), torch.from_numpy(qw).to(DEV), torch.from_numpy(kw).to(DEV)
    ws = B.new_workspace(B.pa_window_workspace_size(R, R, 4 * Hkv, 128, window, sinks), DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.pa_step_tables(new, lens, tables, ring, state, window=window, sink_tokens=sinks, first_page=first, seq_lens=lens,
                         qo_indptr=ind, slot_mapping=slots, positions=pos, free_state_out=state, first_page_out=first,
                         workspace=ws)
        B.pa_qk_norm_rope_append(qkv[:, :4 * Hkv], qkv[:, 4 * Hkv:5 * Hkv], qkv[:, 5 * Hkv:], pos, slots, turns, kc, vc,
                                 q_weight=dqw, k_weight=dkw, q_out=q_out, workspace=ws)
        B.pa_decode_window(q_out, kc, vc, tables, lens, scale, window, sinks, out=out, lse=lse, workspace=ws)
    h = dict(cached=np.zeros(R, np.int32), first=np.zeros(R, np.int32), tables=np.full((R, max_blocks), -1, np.int32),
             ring=np.arange(nb, dtype=np.int32), state=np.array([0, nb], np.int32))
    hk = np.full((nb, Hkv, 16, 128), 0x7fc0, np.uint16)
    hv = hk.copy()
    granted = 0
    for i in range(steps):
        n = np.where((i % 29 == 3) & (np.arange(R) == i % R), -1, 1).astype(np.int32)
        n[R - 1] = i % 2                                     # a request that waits every other step
        x = W.normal_bf16(rng, (R, 6 * Hkv, 128))
        live = n > 0
        m = int(live.sum())
        new.copy_(torch.from_numpy(n))
        qkv[:m].copy_(bf16_dev(x[:m]))                       # the step's tokens side by side
        graph.replay()
        torch.cuda.synchronize()
        t, errors = step.step_tables(n, h["cached"], h["first"], h["tables"], h["ring"], h["state"], window, sinks, 0, R)
        assert not errors and B.pa_get_device_error(ws) == 0, i
        granted += int((-(-(h["cached"] + np.maximum(n, 0)) // 16) - -(-h["cached"] // 16)).sum())
        h = dict(cached=t["seq_lens"], first=t["first_page"], tables=t["block_tables"], ring=t["free_ring"], state=t["free_state"])
        for got, k in ((lens, "cached"), (first, "first"), (tables, "tables"), (ring, "ring"), (state, "state")):
            assert np.array_equal(got.cpu().numpy(), h[k]), (i, k)
        assert np.array_equal(slots.cpu().numpy(), t["slot_mapping"]), i
        # the appended keys are the norm's and rotation's, rounded; the values bit for bit
        s = t["slot_mapping"][:m]
        want, size = step.norm_rope(x[:m, 4 * Hkv:5 * Hkv], kw, t["positions"][:m], f, 1e-6, False)
        got_k = bf16_host(kc)
        err = np.abs(oracle.bf16_to_f64(got_k[s // 16, :, s % 16]) - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size), i
        hk[s // 16, :, s % 16], hv[s // 16, :, s % 16] = got_k[s // 16, :, s % 16], x[:m, 5 * Hkv:]
        assert np.array_equal(got_k, hk) and np.array_equal(bf16_host(vc), hv), i
        if live.all():                                       # row r's query is row r of the step
            q = bf16_host(q_out)
            ref, ref_lse, weight = step.attention_window(q, hk, hv, h["tables"], h["cached"], np.arange(R + 1), scale, window, sinks)
            # as in test_gpu_window.py; |q|_1 max |k| bounds a score's products
            ds = 2.0 ** -16 * scale * np.nanmax(np.abs(oracle.bf16_to_f64(hk))) * np.abs(oracle.bf16_to_f64(q)).sum(-1)
            err = np.abs(oracle.bf16_to_f64(bf16_host(out)) - ref)
            assert np.all(err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 + 4 * ds + 2.0 ** -14)[..., None] * weight), i
            assert np.all(np.abs(lse.cpu().double().numpy() - ref_lse) <= ds + 2.0 ** -20 * (1 + np.abs(ref_lse))), i
    assert granted > nb                                      # some blocks were granted more than once


def test_a_step_with_chunks_and_decode_rows():
    """Tables, then a chunked prompt beside decode rows through the call that
    takes host lengths."""
    Hkv, window, sinks = 2, 100, 4
    cached, n = np.array([300, 0, 500, 77], np.int32), np.array([1, 150, 1, 40], np.int32)
    rng = np.random.default_rng(5)
    had = -(-cached // 16)
    nb = int((-(-(cached + n) // 16)).sum()) + 2
    tables = np.full((4, 40), -1, np.int32)
    perm = rng.permutation(nb).astype(np.int32)
    at = 0
    for r in range(4):
        tables[r, :had[r]] = perm[at:at + had[r]]
        at += had[r]
    ring, state = np.full(nb, -1, np.int32), np.array([0, nb - at], np.int32)
    ring[:nb - at] = perm[at:]
    k, v = W.normal_bf16(rng, (nb, Hkv, 16, 128)), W.normal_bf16(rng, (nb, Hkv, 16, 128))
    N = int(n.sum())
    x = W.normal_bf16(rng, (N, 6 * Hkv, 128))
    f = 1e4 ** (-np.arange(64) / 64)

    def dev(a):
        return torch.from_numpy(a).to(DEV)

    d_tables, kc, vc, qkv = dev(tables), bf16_dev(k), bf16_dev(v), bf16_dev(x)
    ws = B.new_workspace(B.pa_window_workspace_size(4, N, 4 * Hkv, 128, window, sinks), DEV)
    lens, ind, slots, pos, _, _ = B.pa_step_tables(dev(n), dev(cached), d_tables, dev(ring), dev(state), n_tokens=N,
                                                   window=window, sink_tokens=sinks, workspace=ws)
    q = B.pa_qk_norm_rope_append(qkv[:, :4 * Hkv], qkv[:, 4 * Hkv:5 * Hkv], qkv[:, 5 * Hkv:], pos, slots,
                                 B.pa_rope_turns(f).to(DEV), kc, vc, workspace=ws)
    out, lse = B.pa_attention_varlen_window(q, kc, vc, d_tables, lens, ind, 128 ** -0.5, window, sinks,
                                            seq_lens_host=torch.from_numpy(cached + n),
                                            qo_indptr_host=torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)),
                                            workspace=ws, return_lse=True)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    t, _ = step.step_tables(n, cached, np.zeros(4), tables, ring, state, window, sinks, 0, N)
    s = t["slot_mapping"]
    assert np.array_equal(slots.cpu().numpy(), s) and np.array_equal(bf16_host(vc)[s // 16, :, s % 16], x[:, 5 * Hkv:])
    hq, hk = bf16_host(q), bf16_host(kc)
    want, size = step.norm_rope(x[:, :4 * Hkv], None, t["positions"], f, 0, False)
    assert np.all(np.abs(oracle.bf16_to_f64(hq) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size)
    ref, ref_lse, weight = step.attention_window(hq, hk, bf16_host(vc), t["block_tables"], t["seq_lens"], t["qo_indptr"],
                                                 float(np.float32(128 ** -0.5)), window, sinks)
    ds = 2.0 ** -16 * 128 ** -0.5 * np.abs(oracle.bf16_to_f64(hk)).max() * np.abs(oracle.bf16_to_f64(hq)).sum(-1)
    err = np.abs(oracle.bf16_to_f64(bf16_host(out)) - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 4 * ds + 2.0 ** -14)[..., None] * weight)
    assert np.all(np.abs(lse.cpu().double().numpy() - ref_lse) <= ds + 2.0 ** -20 * (1 + np.abs(ref_lse)))
