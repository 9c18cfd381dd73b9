"""What stands around a step's attention, and attention with a window, in plain
64-bit numpy -- TEST INFRASTRUCTURE ONLY.

``step_tables`` walks requests, tokens and pages one at a time; ``norm_rope``
and ``attention_window`` are the formulas in fp64 on bf16 bit patterns.
"""
from __future__ import annotations

import numpy as np

import oracle

PAGE, DIM, GROUP = 16, 128, 4
MAX_LEN = 1 << 20
OK, DEVICE_INDEX, NO_BLOCKS = 0, 5, 7


def step_tables(new, cached, first, tables, ring, state, window, sinks, shared, n_tokens):
    """The tables of a step; tables and ring are copied, not modified.  Returns
    (dict of outputs, set of recorded errors)."""
    tables, ring = tables.copy(), ring.copy()
    R, cap, max_blocks = len(new), len(ring), tables.shape[1]
    head, count = int(state[0]), int(state[1])
    errors = set()
    bound = min(MAX_LEN, max_blocks * PAGE)
    rows = []  # (cached, new, ended, first)
    for r in range(R):
        c, n = int(cached[r]), int(new[r])
        if not 0 <= c <= bound:
            errors.add(DEVICE_INDEX)
            rows.append([0, 0, False, max(int(first[r]), 0)])
            continue
        if c + n > bound:
            errors.add(DEVICE_INDEX)
            n = 0
        rows.append([c, max(n, 0), n < 0, max(int(first[r]), 0)])

    keep = max(-(-sinks // PAGE) if window else 0, shared)

    def returned(c, n, ended, f):
        had = -(-c // PAGE)
        if ended:
            return [j for j in range(had) if j >= shared and (j < keep or j >= f)]
        if window and n > 0:
            return [j for j in range(had) if j >= keep and j >= f and PAGE * (j + 1) <= c - window + 1]
        return []

    back = sum(0 <= tables[r, j] < cap for r, row in enumerate(rows) for j in returned(*row))
    bad = not (0 <= head < cap and 0 <= count <= cap)
    if bad or sum(n for _, n, _, _ in rows) > n_tokens or count + back > cap:
        errors.add(DEVICE_INDEX)
        rows = [[c, 0, False, f] for c, _, _, f in rows]
    seq, indptr, slots, pos, first_out, given_back = [], [0], [], [], [], []
    left, at = (0, 0) if bad else (count, head)
    for r, (c, n, ended, f) in enumerate(rows):
        for j in range(-(-c // PAGE), -(-(c + n) // PAGE)):
            if left > 0:
                block = int(ring[at])
                at, left = (at + 1) % cap, left - 1
                if not 0 <= block < cap:
                    errors.add(DEVICE_INDEX)
                    block = -1
            else:
                errors.add(NO_BLOCKS)
                block = -1
            tables[r, j] = block
        for t in range(c, c + n):
            pos.append(t)
            block = int(tables[r, t // PAGE])
            if block < 0 and t // PAGE < -(-c // PAGE):   # a page that an earlier step could not grant
                errors.add(NO_BLOCKS)
            slots.append(block * PAGE + t % PAGE if block >= 0 else -1)
        out = returned(c, n, ended, f)
        given_back += [int(tables[r, j]) for j in out if 0 <= tables[r, j] < cap]
        seq.append(0 if ended else c + n)
        indptr.append(indptr[-1] + n)
        first_out.append(0 if ended else out[-1] + 1 if out else f)
    if bad:
        at, left = head, count
    else:
        for i, block in enumerate(given_back):
            ring[(head + count + i) % cap] = block
    pad = n_tokens - len(slots)
    i32 = np.int32
    return dict(seq_lens=np.array(seq, i32), qo_indptr=np.array(indptr, i32),
                slot_mapping=np.array(slots + [-1] * pad, np.int64), positions=np.array(pos + [0] * pad, i32),
                free_state=np.array([at, left + len(given_back)], i32), first_page=np.array(first_out, i32),
                block_tables=tables, free_ring=ring), errors


def norm_rope(x, weight, positions, inv_freq, eps, interleaved):
    """fp64 [N, H, 128] from bf16 bits x, and a bound on the size of what each
    result is the sum of (|a| + |b| of its pair)."""
    y = oracle.bf16_to_f64(x)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    h = len(inv_freq)
    i = np.arange(h)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    t = positions.astype(np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    a, b = y[..., ia], y[..., ib]
    out, size = y.copy(), np.abs(y)
    out[..., ia], out[..., ib] = a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return out, size


def attention_window(q, k_cache, v_cache, tables, seq_lens, qo_indptr, sm_scale, window, sinks):
    """fp64 (out, lse, sum_t p_t |v_t|) of bf16 bits; every query's keys are
    gathered for it alone."""
    q, total = oracle.bf16_to_f64(q), q.shape[0]
    H = k_cache.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    for r in range(len(seq_lens)):
        n = int(qo_indptr[r + 1] - qo_indptr[r])
        for j in range(n):
            p, i = int(seq_lens[r]) - n + j, int(qo_indptr[r]) + j
            t = np.arange(p + 1)
            t = t[(t < sinks) | (t > p - window)]
            block = tables[r, t // PAGE].astype(np.int64)
            ok = (block >= 0) & (block < k_cache.shape[0])
            t, block = t[ok], block[ok]
            if not len(t):
                continue
            k = oracle.bf16_to_f64(k_cache[block, :, t % PAGE])     # [T, H, 128]
            v = oracle.bf16_to_f64(v_cache[block, :, t % PAGE])
            s = np.einsum("hgd,thd->hgt", q[i].reshape(H, GROUP, DIM), k) * sm_scale
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            l = w.sum(-1, keepdims=True)
            out[i] = np.einsum("hgt,thd->hgd", w / l, v).reshape(-1, DIM)
            size[i] = np.einsum("hgt,thd->hgd", w / l, np.abs(v)).reshape(-1, DIM)
            lse[i] = (m + np.log(l))[..., 0].reshape(-1)
    return out, lse, size
