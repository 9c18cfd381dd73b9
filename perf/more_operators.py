"""Timed cases of what stands around a serving step's attention, and of its
form with a sliding window.

A case is a dict of plain values.  `op` says which path it takes:

  tables  block tables, slots, positions and query offsets of a step, from the
          requests' lengths: pages come from a ring of free blocks, those
          behind the window or of ended requests go back to it
  rope    queries and keys normalised per head and rotated by their positions;
          with `append`, keys and values go to their slots of the bf16 pools
  window  a batch of rows attends to the last `window` keys of its cached
          tokens and to their first `sinks`
  step    one layer of a serving step with such a window: tables, rope with
          append, attention

Layouts are those of the library: pools [num_blocks, kv_heads, 16, 128] bf16,
block tables [rows, max_blocks] int32, 4 query heads per kv head.
"""
import math

import torch

own = False

DIM, PAGE, QPK = 128, 16, 4
EPS = 1e-6


def _tables(name, rows, lo, hi, new_lo=1, new_hi=1, q_rows=0, idle=0, ended=0, window=0, sinks=0, shared=0):
    """rows requests with lo .. hi cached tokens; the first q_rows of them (0: all)
    bring new_lo .. new_hi new tokens, the others one; every idle-th none, and
    every ended-th ends."""
    return dict(name=name, op="tables", rows=rows, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, q_rows=q_rows,
                idle=idle, ended=ended, window=window, sinks=sinks, shared=shared)


def _rope(name, tokens, kv_heads=8, far=4096, rotary=128, interleaved=False, base=1e6, append=True, norm=True, fused=True,
          skip=0):
    """tokens at positions below far; fused: q, k and v are columns of one product's
    rows; every skip-th token is padding."""
    return dict(name=name, op="rope", kv_heads=kv_heads, tokens=tokens, far=far, rotary=rotary, interleaved=interleaved,
                base=base, append=append, norm=norm, fused=fused, skip=skip)


def _window(name, rows, lo, hi, window, sinks=0, q=1, q_rows=0, empty=0, kv_heads=8, op="window"):
    """rows requests of lo .. hi tokens; the first q_rows of them (0: all) bring q
    queries (-1: as many as they have tokens), the others one; every empty-th
    one brings none."""
    return dict(name=name, op=op, kv_heads=kv_heads, rows=rows, lo=lo, hi=hi, window=window, sinks=sinks, q=q,
                q_rows=q_rows, empty=empty)


def listed():
    return [
        # a decode step of 64 requests: four of them cross into a new page: latency
        _tables("tables decode step", 64, 500, 9000),
        # 1000 requests, some waiting, some done, prompts coming in by chunks, behind a window
        _tables("tables busy step", 1000, 0, 30000, 30, 1100, q_rows=14, idle=9, ended=31, window=4096, sinks=4),
        # one decode step's new tokens for 64 requests: latency
        _rope("rope 64 new tokens", 64),
        # a prefill chunk of 8 Ki tokens, some of them padding
        _rope("rope a prefill chunk", 8191, skip=7),
        # keys for a 4-bit pool: rotated pairwise in half their dims, far into a context, not appended
        _rope("rope far positions", 1000, far=1000000, rotary=64, interleaved=True, base=5e5, append=False, fused=False),
        # a handful of short requests: latency
        _window("window few short rows", 4, 17, 1500, 256, 4),
        # 64 long conversations behind a window
        _window("window decode batch", 64, 3000, 30000, 1024, 4),
        # few rows with a wide window: the work has to be split over the keys
        _window("window wide decode", 3, 40000, 90000, 32768, 16),
        # speculative verification: 5 query tokens over ragged rows, some of them waiting
        _window("window verify rows", 80, 300, 9000, 1024, 4, q=5, empty=9),
        # chunked prefill late in long prompts: bound by the products
        _window("window late chunks", 4, 6000, 12000, 4096, 4, q=512),
        # whole prompts of odd lengths in one pass, a narrow window
        _window("window whole prompts", 8, 100, 3000, 512, 0, q=-1),
        # a decode step's layer: tables, norms, rotations and append, attention
        _window("step decode layer", 64, 2000, 20000, 1024, 4, op="step"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "window", "window", "window", "step"])
    if op == "tables":
        rows = _log(rng, 1, 3000)
        c = _tables("", rows, rng.choice([0, 1, 100]), _log(rng, 100, 30000), 1, _log(rng, 1, 1200),
                    q_rows=rng.randint(1, min(rows, 14)), idle=rng.choice([0, 0, 3, 11]), ended=rng.choice([0, 0, 5, 40]),
                    window=rng.choice([0, 0, _log(rng, 16, 8000)]), sinks=rng.choice([0, 4, 20]), shared=rng.choice([0, 0, 3]))
    elif op == "rope":
        inter = rng.random() < 0.3
        c = _rope("", _log(rng, 1, 8000), rng.choice([8, 8, 2, 1, 5]), _log(rng, 64, 1000000),
                  rng.choice([128, 128, 64, 32, 96]), inter, rng.choice([1e4, 5e5, 1e6]), rng.random() < 0.7,
                  rng.random() < 0.8, rng.random() < 0.6, rng.choice([0, 0, 2, 11]))
    else:
        kind = rng.choice(["decode", "decode", "verify", "chunk", "mixed"]) if op == "window" else "decode"
        kv_heads = rng.choice([8, 8, 4, 2, 1, 3]) if op == "window" else rng.choice([8, 8, 2, 1, 5])
        sinks = rng.choice([0, 0, 1, 4, 16, 70])
        empty = rng.choice([0, 0, 3, 8])
        if kind in ("decode", "verify"):
            rows = _log(rng, 1, 300)
            window = _log(rng, 8, min(32768, 60000 // rows))
            hi = _log(rng, 30, min(90000, 1500000 // rows))
            c = _window("", rows, max(1, int(hi * rng.random())), hi, window, sinks,
                        1 if kind == "decode" else rng.randint(2, 9), 0, empty if op == "window" else 0, kv_heads, op)
        else:
            rows = rng.randint(1, 3) if kind == "chunk" else rng.randint(2, 12)
            hi = _log(rng, 40, 8000)
            c = _window("", rows, max(1, int(hi * rng.random())), hi, _log(rng, 16, 4096), sinks, rng.randint(10, 400),
                        0 if kind == "chunk" else 1, empty if rows > 3 else 0, kv_heads)
    del c["name"]
    return c


# --------------------------------------------------------------- plain forms
def _step_tables(s):
    """The step's tables from new_tokens (negative: the request ends) and
    cached_lens."""
    new, cached, first, tables = s["new_tokens"].long(), s["cached_lens"].long(), s["first_page"].long(), s["block_tables"]
    ring, (window, sinks, shared) = s["free_ring"], s["rule"]
    dev, cap, n_tok = new.device, ring.shape[0], s["n_tokens"]
    head, count = s["free_state"].long()
    n, ended = new.clamp(min=0), new < 0
    had, has = (cached + PAGE - 1) // PAGE, (cached + n + PAGE - 1) // PAGE
    indptr = torch.zeros(new.shape[0] + 1, dtype=torch.int64, device=dev)
    indptr[1:] = torch.cumsum(n, 0)

    def ragged(lo, hi):
        """Rows and values of lo[r] .. hi[r] - 1 for every r, one after another."""
        size = (hi - lo).clamp(min=0)
        row = torch.repeat_interleave(torch.arange(size.shape[0], device=dev), size)
        return row, lo[row] + torch.arange(row.shape[0], device=dev) - (torch.cumsum(size, 0) - size)[row]

    # pages granted, in the order of requests
    row, page = ragged(had, torch.where(ended, had, has))
    tables[row, page] = ring[(head + torch.arange(row.shape[0], device=dev)) % cap]
    granted = row.shape[0]
    # pages given back: of an ended request those before `keep` first
    keep = max((sinks + PAGE - 1) // PAGE if window else 0, shared)
    from_ = torch.where(first > keep, first, torch.full_like(first, keep))
    upto = torch.minimum((cached - window + 1).clamp(min=0) // PAGE, had)
    moved = (n > 0) & (upto > from_) & (window > 0)
    none = torch.zeros_like(had)
    lo = torch.stack([torch.where(ended, shared + none, none), from_], 1)
    hi = torch.stack([torch.where(ended, had.clamp(max=keep), none), torch.where(ended, had, torch.where(moved, upto, none))], 1)
    row, page = ragged(lo.flatten(), hi.flatten())
    back = tables[row // 2, page]
    ring[(head + count + torch.arange(row.shape[0], device=dev)) % cap] = back
    state = torch.stack([(head + granted) % cap, count - granted + row.shape[0]]).to(torch.int32)
    lens = torch.where(ended, none, cached + n)
    new_first = torch.where(ended, none, torch.where(moved, upto, first))
    slots = torch.full((n_tok,), -1, dtype=torch.int64, device=dev)
    positions = torch.zeros(n_tok, dtype=torch.int32, device=dev)
    row, pos = ragged(cached, cached + n)
    positions[:row.shape[0]] = pos.to(torch.int32)
    slots[:row.shape[0]] = tables[row, pos // PAGE].long() * PAGE + pos % PAGE
    return dict(seq_lens=lens.to(torch.int32), qo_indptr=indptr.to(torch.int32), slot_mapping=slots, positions=positions,
                free_state=state, first_page=new_first.to(torch.int32), block_tables=tables, free_ring=ring)


def _norm_rope(x, weight, cos, sin, interleaved):
    """Heads x [n, H, 128], normalised with weight (None: not), the first dims
    rotated by the angles of cos / sin [n, rotary / 2]."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    h = cos.shape[1]
    rot, rest = y[..., :2 * h], y[..., 2 * h:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :h], rot[..., h:])
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    rot = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([rot, rest], -1).bfloat16()


def _rope_append(s, positions, slots):
    angle = positions.double()[:, None] * s["inv_freq"][None, :]     # far positions: in 64 bits
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _norm_rope(s["q"], s["q_weight"], cos, sin, s["interleaved"])
    k = _norm_rope(s["k"], s["k_weight"], cos, sin, s["interleaved"])
    if slots is None:
        return q, k
    at = torch.nonzero(slots >= 0)[:, 0]
    block, off = slots[at] // PAGE, slots[at] % PAGE
    s["k_cache"][block, :, off] = k[at]
    s["v_cache"][block, :, off] = s["v"][at]
    return q


def _attend(s, q, tables, seq_lens, qo_indptr):
    """Softmax attention of every row over its first tokens and its window,
    padded to the row with the most pages."""
    window, sinks = s["rule"][:2]
    indptr, lens = qo_indptr.long(), seq_lens.long()
    n = indptr[1:] - indptr[:-1]
    start = lens - n                                                 # position of a row's first query
    pages = (lens + PAGE - 1) // PAGE
    lead = pages.clamp(max=(sinks + PAGE - 1) // PAGE)
    first = torch.maximum((start - window + 1).clamp(min=0) // PAGE, lead)
    v = torch.arange(s["max_pages"], device=q.device)
    page = torch.where(v < lead[:, None], v, v + (first - lead)[:, None])
    there = page < pages[:, None]
    ids = torch.gather(tables, 1, torch.where(there, page, 0)).clamp(min=0).long()
    K, V = (s[c][torch.where(there, ids, 0)].transpose(1, 2).flatten(2, 3).float() for c in ("k_cache", "v_cache"))
    pos = (page[:, :, None] * PAGE + torch.arange(PAGE, device=q.device)).flatten(1)  # [R, T]
    R, H, T = K.shape[:3]
    tok = torch.arange(q.shape[0], device=q.device)
    r = torch.searchsorted(indptr, tok, right=True) - 1
    j = tok - indptr[r]
    n_q = s["max_q"]
    Q = torch.zeros(R, n_q, H * QPK, DIM, device=q.device)
    Q[r, j] = q.float()
    Q = Q.reshape(R, n_q, H, QPK, DIM).permute(0, 2, 1, 3, 4).reshape(R, H, n_q * QPK, DIM)
    sc = (Q @ K.transpose(-1, -2)).mul_(s["sm_scale"])
    at = (start[:, None] + torch.arange(n_q, device=q.device))[:, :, None]
    seen = (pos[:, None] <= at) & ((pos[:, None] < sinks) | (pos[:, None] > at - window)) & (pos < lens[:, None])[:, None]
    sc.masked_fill_(~seen.repeat_interleave(QPK, 1)[:, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ V) / l
    lse = m + torch.log(l)
    o = o.reshape(R, H, n_q, QPK, DIM).transpose(1, 2).reshape(R, n_q, H * QPK, DIM)[r, j]
    lse = lse.reshape(R, H, n_q, QPK).transpose(1, 2).reshape(R, n_q, H * QPK)[r, j]
    return o.bfloat16(), lse


# ---------------------------------------------------------------------- cases
def _counts(case):
    """Cached tokens and new tokens of every row: the case's own, whatever the
    seed.  tables: -1 for a request that ends."""
    R = case["rows"]
    gen = torch.Generator().manual_seed(R * 1000003 + case["lo"] * 1009 + case["hi"])
    lens = torch.randint(case["lo"], case["hi"] + 1, (R,), generator=gen)
    n = torch.ones(R, dtype=torch.int64)
    many = R if case["q_rows"] == 0 else case["q_rows"]
    if case["op"] == "tables":
        n[:many] = torch.randint(case["new_lo"], case["new_hi"] + 1, (many,), generator=gen)
        if case["idle"]:
            n[case["idle"] - 1::case["idle"]] = 0
        if case["ended"]:
            n[case["ended"] - 1::case["ended"]] = -1
        return lens, n
    n[:many] = lens[:many] if case["q"] < 0 else torch.minimum(lens[:many], torch.tensor(case["q"]))
    if case["empty"]:
        n[case["empty"] - 1::case["empty"]] = 0
    return lens - n, n


def _normal(gen, shape, device, spread=0.0):
    """Normal values; spread: each of the last dims with a scale of its own."""
    x = torch.randn(shape, generator=gen, device=device)
    if spread:
        x *= torch.exp(spread * torch.randn(shape[1:], generator=gen, device=device))
    return x.bfloat16()


def _visible(case, cached, n):
    """Pages of each row that its queries see: leading ones, the first behind
    them, and the end."""
    pages = (cached + n + PAGE - 1) // PAGE
    lead = pages.clamp(max=-(-case["sinks"] // PAGE))
    first = torch.maximum((cached - case["window"] + 1).clamp(min=0) // PAGE, lead)
    return lead, torch.minimum(first, pages), pages


def _pages(case, cached, n, host, dev, s):
    """Block tables, free ring and what goes with them, before the step: every
    row holds the pages that its last step left it."""
    R = case["rows"]
    window, shared = case["window"], case.get("shared", 0)
    keep = max(-(-case["sinks"] // PAGE) if window else 0, shared)
    had, has = (cached + PAGE - 1) // PAGE, (cached + n.clamp(min=0) + PAGE - 1) // PAGE
    first = torch.zeros_like(had)
    if window:  # the step before began a token earlier
        upto = (cached - window).clamp(min=0) // PAGE
        first = torch.where(upto > keep, upto, first)
    col = torch.arange(int(has.max()) + 2)
    held = (col < had[:, None]) & ((col < keep) | (col >= first[:, None]))
    blocks = int(held.sum()) + int((has - had).clamp(min=0).sum()) + 5
    perm = torch.randperm(blocks, generator=host).to(torch.int32)
    tables = torch.full(held.shape, -1, dtype=torch.int32)
    tables[held] = perm[:int(held.sum())]
    free = perm[int(held.sum()):]
    head = int(torch.randint(0, blocks, (1,), generator=host))
    ring = torch.full((blocks,), -1, dtype=torch.int32)
    ring[(head + torch.arange(free.shape[0])) % blocks] = free
    total = int(n.clamp(min=0).sum())
    s.update(new_tokens=n.to(torch.int32).to(dev), cached_lens=cached.to(torch.int32).to(dev),
             first_page=first.to(torch.int32).to(dev), block_tables=tables.to(dev), free_ring=ring.to(dev),
             free_state=torch.tensor([head, free.shape[0]], dtype=torch.int32).to(dev),
             rule=(window, case["sinks"], shared), n_tokens=total + (5 if case["op"] == "tables" else 0))
    return blocks, total


def prepare(case, seed):
    """What a serving loop holds before the call: its pools, tables and
    metadata, the layer's q, k, v and weights, and the buffers it keeps."""
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = dict(op=case["op"])
    i32 = dict(dtype=torch.int32, device=dev)
    if case["op"] in ("tables", "step"):
        cached, n = _counts(case)
        blocks, tokens = _pages(case, cached, n, host, dev, s)
        s["out"] = dict(seq_lens=torch.empty(case["rows"], **i32), qo_indptr=torch.empty(case["rows"] + 1, **i32),
                        slot_mapping=torch.empty(s["n_tokens"], dtype=torch.int64, device=dev),
                        positions=torch.empty(s["n_tokens"], **i32), free_state_out=torch.empty(2, **i32),
                        first_page_out=torch.empty(case["rows"], **i32))
    if case["op"] in ("rope", "step"):
        H = case["kv_heads"]
        rotary, base, fused, norm, skip = (case.get(k, d) for k, d in (
            ("rotary", DIM), ("base", 1e6), ("fused", True), ("norm", True), ("skip", 0)))
        if case["op"] == "rope":
            tokens = case["tokens"]
            s["positions"] = torch.randint(0, case["far"], (tokens,), generator=host).to(torch.int32).to(dev)
            blocks = -(-tokens // PAGE) + 3
            if case["append"]:
                slots = torch.randperm(blocks * PAGE, generator=host)[:tokens]
                if tokens > 1000:               # long stretches lie in pages of one request each
                    page = torch.randperm(blocks, generator=host)[:-(-tokens // PAGE)]
                    slots = (page[:, None] * PAGE + torch.arange(PAGE)).flatten()[:tokens].contiguous()
                if skip:
                    slots[skip - 1::skip] = -1
                s["slot_mapping"] = slots.to(dev)
        s["interleaved"] = case.get("interleaved", False)
        if fused:
            qkv = _normal(gen, (tokens, (QPK + 2) * H * DIM), dev, 0.4).reshape(tokens, (QPK + 2) * H, DIM)
            q, k, v = qkv[:, :QPK * H], qkv[:, QPK * H:QPK * H + H], qkv[:, QPK * H + H:]
        else:
            q, k, v = (_normal(gen, (tokens, h, DIM), dev, 0.4) for h in (QPK * H, H, H))
        s.update(q=q, k=k, v=v, inv_freq=base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary).to(dev))
        for name in ("q_weight", "k_weight"):
            s[name] = 1 + 0.3 * torch.randn(DIM, generator=gen, device=dev) if norm else None
        s["q_out"] = torch.empty(tokens, QPK * H, DIM, dtype=torch.bfloat16, device=dev)
        if case["op"] == "rope" and case["append"]:
            s["k_cache"] = torch.zeros(blocks, H, PAGE, DIM, dtype=torch.bfloat16, device=dev)
            s["v_cache"] = torch.zeros_like(s["k_cache"])
        elif case["op"] == "rope":
            s["k_out"] = torch.empty(tokens, H, DIM, dtype=torch.bfloat16, device=dev)
    if case["op"] in ("window", "step"):
        H, R = case["kv_heads"], case["rows"]
        cached, n = _counts(case)
        lens = cached + n
        lead, first, pages = _visible(case, cached, n)
        total = int(n.sum())
        if case["op"] == "window":
            col = torch.arange(int(pages.max()))
            held = (col < pages[:, None]) & ((col < lead[:, None]) | (col >= first[:, None])) & (n > 0)[:, None]
            blocks = int(held.sum()) + 3
            tables = torch.full(held.shape, -1, dtype=torch.int32)   # pages that no query sees are gone
            tables[held] = torch.randperm(blocks, generator=host)[:int(held.sum())].to(torch.int32)
            indptr = torch.zeros(R + 1, dtype=torch.int32)
            indptr[1:] = torch.cumsum(n, 0)
            s.update(tables=tables.to(dev), seq_lens=lens.to(torch.int32).to(dev), qo_indptr=indptr.to(dev),
                     seq_lens_host=lens.to(torch.int32), qo_indptr_host=indptr,
                     q=_normal(gen, (total, H * QPK, DIM), dev), rule=(case["window"], case["sinks"]))
        shape = (blocks, H, PAGE, DIM)
        s["k_cache"], s["v_cache"] = _normal(gen, shape, dev), _normal(gen, shape, dev)
        s.update(sm_scale=1.0 / math.sqrt(DIM), max_q=int(n.max()), max_pages=int((lead + pages - first).max()),
                 attn=torch.empty(total, H * QPK, DIM, dtype=torch.bfloat16, device=dev),
                 lse=torch.empty(total, H * QPK, dtype=torch.float32, device=dev))
    if own:
        from paged_kv_decode_varlen_gb300 import binding as B
        s["binding"] = B
        size = B.PA_ERROR_WORD_BYTES
        if case["op"] in ("window", "step"):
            size = B.pa_window_workspace_size(case["rows"], total, H * QPK, DIM, case["window"], case["sinks"])
        s["workspace"] = B.new_workspace(size, dev)
        if "inv_freq" in s:
            s["turns"] = B.pa_rope_turns(s["inv_freq"].cpu()).to(dev)
    return s


def _own_tables(B, s):
    window, sinks, shared = s["rule"]
    o = s["out"]
    B.pa_step_tables(s["new_tokens"], s["cached_lens"], s["block_tables"], s["free_ring"], s["free_state"],
                     window=window, sink_tokens=sinks, shared_pages=shared, first_page=s["first_page"],
                     workspace=s["workspace"], **o)
    return dict(seq_lens=o["seq_lens"], qo_indptr=o["qo_indptr"], slot_mapping=o["slot_mapping"], positions=o["positions"],
                free_state=o["free_state_out"], first_page=o["first_page_out"], block_tables=s["block_tables"],
                free_ring=s["free_ring"])


def run(s):
    op = s["op"]
    if own:
        B, ws = s["binding"], s["workspace"]
        if op in ("tables", "step"):
            t = _own_tables(B, s)
        if op == "tables":
            return t
        if op == "rope" and "k_out" in s:
            return B.pa_qk_norm_rope(s["q"], s["k"], s["positions"], s["turns"], q_weight=s["q_weight"],
                                     k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"], q_out=s["q_out"],
                                     k_out=s["k_out"])
        if op in ("rope", "step"):
            where = s if op == "rope" else t
            q = B.pa_qk_norm_rope_append(s["q"], s["k"], s["v"], where["positions"], where["slot_mapping"], s["turns"],
                                         s["k_cache"], s["v_cache"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                         interleaved=s["interleaved"], q_out=s["q_out"], workspace=ws)
        if op == "rope":
            return q, s["k_cache"], s["v_cache"]
        if op == "step":
            out, lse = B.pa_decode_window(q, s["k_cache"], s["v_cache"], t["block_tables"], t["seq_lens"], s["sm_scale"],
                                          *s["rule"][:2], out=s["attn"], lse=s["lse"], workspace=ws)
            return t, q, s["k_cache"], s["v_cache"], out, lse
        return B.pa_attention_varlen_window(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"], s["qo_indptr"],
                                            s["sm_scale"], *s["rule"], seq_lens_host=s["seq_lens_host"],
                                            qo_indptr_host=s["qo_indptr_host"], out=s["attn"], lse=s["lse"], workspace=ws)
    if op == "tables":
        return _step_tables(s)
    if op == "rope":
        if "k_out" in s:
            return _rope_append(s, s["positions"], None)
        return _rope_append(s, s["positions"], s["slot_mapping"]), s["k_cache"], s["v_cache"]
    if op == "step":
        t = _step_tables(s)
        q = _rope_append(s, t["positions"], t["slot_mapping"])
        return t, q, s["k_cache"], s["v_cache"], *_attend(s, q, t["block_tables"], t["seq_lens"], t["qo_indptr"])
    return _attend(s, s["q"], s["tables"], s["seq_lens"], s["qo_indptr"])


def work(case):
    """Bytes: each input once, each output once (a row's visible tokens are
    read once, whatever the number of its queries).  Flops: the two products."""
    b = flops = 0
    if case["op"] in ("tables", "step"):
        cached, n = _counts(case)
        new = n.clamp(min=0)
        granted = int(((cached + new + PAGE - 1) // PAGE - (cached + PAGE - 1) // PAGE).sum())
        b += case["rows"] * 24 + int(new.sum()) * 12 + granted * 8
    if case["op"] in ("rope", "step"):
        H = case["kv_heads"]
        tokens = case["tokens"] if case["op"] == "rope" else int(n.sum())
        skip = case.get("skip", 0)
        live = tokens - (tokens // skip if skip else 0)
        b += tokens * (QPK * H * DIM * 4 + 4)                       # q in and out, positions
        if case.get("append", True):
            b += tokens * 8 + live * 2 * H * DIM * 4                # slots; k and v in and out
        else:
            b += tokens * H * DIM * 4
    if case["op"] in ("window", "step"):
        H, W, S = case["kv_heads"], case["window"], case["sinks"]
        cached, n = _counts(case)
        lens, total = cached + n, int(n.sum())
        low = (cached - W + 1).clamp(min=0)
        tokens = torch.where(n > 0, lens - low + torch.minimum(low, torch.tensor(S)), 0)
        b += int(tokens.sum()) * 4 * H * DIM + int((tokens // PAGE + 1).sum()) * 4
        b += total * H * QPK * (4 * DIM + 4) + 8 * case["rows"] + 4
        p = torch.repeat_interleave(cached, n) + torch.cat([torch.arange(int(k)) for k in n])
        low = (p - W + 1).clamp(min=0)
        flops = 4 * DIM * QPK * H * int((p + 1 - low + low.clamp(max=S)).sum())
    return {"bytes": b, "flops": flops}


# ------------------------------------------------------- the definition in 64 bits
def _exact_rotated(x, weight, positions, inv_freq, interleaved):
    """Each pair of dims as a complex number, turned."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(torch.sum(y ** 2, -1, keepdim=True) / DIM + EPS) * weight.double()
    h = inv_freq.shape[0]
    re = torch.arange(h, device=x.device) * (2 if interleaved else 1)
    im = re + (1 if interleaved else h)
    angle = torch.outer(positions.double(), inv_freq.double())
    z = torch.complex(y[..., re], y[..., im]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y = y.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_attention(q, k_cache, v_cache, rows, sm_scale, window, sinks):
    """rows: (first query, queries, tokens, table) of each request; the pools
    as dicts of float64 pages by block or as tensors."""
    outs, lses = [], []
    H = k_cache.shape[1]
    for q0, n, L, table in rows:
        if n == 0:
            continue
        p = L - n + torch.arange(n, device=q.device)
        t = torch.arange(L, device=q.device)
        t = t[(t < sinks) | (t > L - n - window)]
        block = table.long()[t // PAGE]
        k, v = (c[block, :, t % PAGE].double() for c in (k_cache, v_cache))
        sc = torch.einsum("nhgd,thd->nhgt", q[q0:q0 + n].double().reshape(n, H, QPK, DIM), k) * sm_scale
        hidden = (t[None] > p[:, None]) | ((t[None] >= sinks) & (t[None] <= p[:, None] - window))
        sc = sc.masked_fill(hidden[:, None, None], -math.inf)
        outs.append(torch.einsum("nhgt,thd->nhgd", torch.softmax(sc, -1), v).reshape(n, H * QPK, DIM))
        lses.append(torch.logsumexp(sc, -1).reshape(n, H * QPK))
    return torch.cat(outs), torch.cat(lses)


def exact(case, seed):
    if case["op"] == "tables":
        return None                                                 # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "window":
        ind = s["qo_indptr_host"].tolist()
        rows = [(ind[r], ind[r + 1] - ind[r], int(s["seq_lens_host"][r]), s["tables"][r]) for r in range(case["rows"])]
        return _exact_attention(s["q"], s["k_cache"], s["v_cache"], rows, s["sm_scale"], case["window"], case["sinks"])
    if case["op"] == "rope":
        q, k = (_exact_rotated(s[x], s[x + "_weight"], s["positions"], s["inv_freq"], s["interleaved"]) for x in ("q", "k"))
        if not case["append"]:
            return q, k
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for i, slot in enumerate(s["slot_mapping"].tolist()):
            if slot >= 0:
                kc[slot // PAGE, :, slot % PAGE] = k[i]
                vc[slot // PAGE, :, slot % PAGE] = s["v"][i].double()
        return q, kc, vc
    # step: a token for each row, its page taken from the ring where the last one is full
    cached = s["cached_lens"].tolist()
    pos = torch.tensor(cached, device=s["q"].device)
    q, k = (_exact_rotated(s[x], s[x + "_weight"], pos, s["inv_freq"], s["interleaved"]) for x in ("q", "k"))
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    ring, (at, _) = s["free_ring"].tolist(), s["free_state"].tolist()
    rows = []
    for r, c in enumerate(cached):
        table = s["block_tables"][r].clone()
        if c % PAGE == 0:
            table[c // PAGE] = ring[at % len(ring)]
            at += 1
        block = int(table[c // PAGE])
        kc[block, :, c % PAGE], vc[block, :, c % PAGE] = k[r], s["v"][r].double()
        rows.append((r, 1, c + 1, table))
    # what the attention reads was rounded to bf16 as it was written
    out, lse = _exact_attention(q.bfloat16(), kc.bfloat16(), vc, rows, s["sm_scale"], case["window"], case["sinks"])
    return None, q, kc, vc, out, lse
