"""Timed cases of the 4-bit KV cache: quantising keys and values as they are
written, reading them back, and attention over the 4-bit pages.

A case is a dict of plain values.  `op` says which path it takes:

  write      new tokens are quantised into their slots and those slots read
             back as bf16 rows (what leaves for another worker, or is promoted
             to a bf16 pool)
  read       cached tokens are read back as bf16 rows by their slots
  attention  a batch of rows attends to its cached tokens through block tables
  step       one layer of a serving step: the batch's new tokens are appended,
             then attended to together with the cached ones

A 4-bit pool is uint8 [num_blocks, kv_heads, 1280].  A slab holds 16 tokens:
64 bytes of codes per token (group g of 32 dims at 16 (g ^ ((t >> 1) & 3)),
8 dims per 32-bit word, even dims in its low half, odd dims in its high half),
then per token and group two bf16, D and Z.  A code c stands for the bf16
nearest to Z + D (1 + c / 16).  Every row has 4 query heads per kv head and
128 dims per head.
"""
import math

import torch

own = False

DIM, PAGE, GROUP, QPK = 128, 16, 32, 4
CODES = PAGE * DIM // 2             # 1024 bytes of codes in a slab
SLAB = CODES + PAGE * DIM // GROUP * 4  # then (D, Z) pairs: 1280


def _case(name, op, kv_heads=8, tokens=0, skip=0, rows=0, lo=0, hi=0, q=1, q_rows=0, empty=0):
    """tokens / skip: tokens written or read, every skip-th of them padding.
    rows: requests of lo .. hi tokens; the first q_rows of them (0: all) bring
    q queries (-1: as many as they have tokens), the others one; every
    empty-th one brings none."""
    c = dict(op=op, kv_heads=kv_heads)
    if op in ("write", "read"):
        c.update(tokens=tokens, skip=skip)
    else:
        c.update(rows=rows, lo=lo, hi=hi, q=q, q_rows=q_rows, empty=empty)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's new tokens for 64 requests: latency
        _case("write 64 new tokens", "write", tokens=64),
        # a prefill chunk of 8 Ki tokens, some of them padding
        _case("write a prefill chunk", "write", tokens=8191, skip=7),
        # a prompt handed to another worker
        _case("read a prompt", "read", tokens=1000),
        # a long context promoted to bf16
        _case("read a long context", "read", tokens=131072),
        # the short-dialogue decode step: 64 requests of 2.0-2.3K tokens
        _case("step short dialogue", "step", rows=64, lo=2048, hi=2303),
        # a handful of short requests: latency
        _case("decode few short rows", "attention", rows=4, lo=17, hi=513),
        # one request with a long context: the work has to be split over its keys
        _case("decode one long row", "attention", rows=1, lo=131072, hi=131072),
        # many ragged requests, some of them waiting, on a model with 4 kv heads
        _case("decode ragged rows", "attention", kv_heads=4, rows=200, lo=1, hi=1500, empty=9),
        # speculative verification: 5 query tokens over each short dialogue
        _case("step verify rows", "step", rows=64, lo=2048, hi=2303, q=5),
        # chunked prefill late in long prompts: bound by the products
        _case("prefill late chunks", "attention", rows=4, lo=4096, hi=8192, q=512),
        # a mixed step: 32 decode rows and one chunk of 512
        _case("step mixed batch", "step", rows=33, lo=2048, hi=4096, q=512, q_rows=1),
        # whole prompts of odd lengths in one pass, nothing cached before
        _case("prefill whole prompts", "attention", rows=8, lo=100, hi=1000, q=-1),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "step", "step"])
    kv_heads = rng.choice([8, 8, 4, 2, 1, 3])
    if op in ("write", "read"):
        return _case("", op, kv_heads, tokens=_log(rng, 1, 60000), skip=rng.choice([0, 0, 2, 5, 11]))
    kind = rng.choice(["decode", "decode", "verify", "chunk", "mixed"])
    empty = rng.choice([0, 0, 3, 8])
    if kind in ("decode", "verify"):
        rows = _log(rng, 1, 300)
        hi = _log(rng, 16, min(100000, 150000 // rows))
        return _case("", op, kv_heads, rows=rows, lo=max(1, int(hi * rng.random())), hi=hi,
                     q=1 if kind == "decode" else rng.randint(2, 9), empty=empty)
    rows = rng.randint(1, 3) if kind == "chunk" else rng.randint(2, 12)
    hi = _log(rng, 40, 6000)
    return _case("", op, kv_heads, rows=rows, lo=max(1, int(hi * rng.random())), hi=hi, q=rng.randint(10, 400),
                 q_rows=0 if kind == "chunk" else 1, empty=empty if rows > 3 else 0)


# ----------------------------------------------------------------- plain form
def _quantise(x):
    """bf16 [..., 128] -> codes int32 [..., 4, 32], (D, Z) bf16 [..., 4, 2]."""
    v = x.float().reshape(*x.shape[:-1], DIM // GROUP, GROUP)
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    d = ((hi - lo) / 15.0 * 16.0).bfloat16()
    z = (lo - d.float()).bfloat16()
    df, zf = d.float(), z.float()
    c = torch.round((v - zf) / torch.where(df == 0, torch.ones_like(df), df) * 16.0 - 16.0).clamp(0, 15)
    c = torch.where(df == 0, torch.zeros_like(c), c)
    return c.to(torch.int32), torch.cat([d, z], -1)


def _seats(off):
    """Token offsets [n] in their pages -> the byte of each group's codes [n, 4]."""
    g = torch.arange(DIM // GROUP, device=off.device)
    return 64 * off[:, None] + 16 * (g[None, :] ^ ((off[:, None] >> 1) & 3))


def _store(x, slots, pool):
    """Quantises rows x [n, H, 128] into their slots (negative: padding)."""
    keep = torch.nonzero(slots >= 0)[:, 0]
    slot = slots[keep]
    c, dz = _quantise(x[keep])
    n, H = c.shape[:2]
    # word w of a group: dim 8 w + 2 i + e at bits 16 e + 4 i, as bytes (e, i / 2)
    c = c.reshape(n, H, 4, 4, 2, 2, 2)          # [.., g, w, i / 2, i % 2, e]
    by = (c[..., 0, :] | (c[..., 1, :] << 4)).transpose(-1, -2).reshape(n, H, 4, 16).to(torch.uint8)
    blk, off = slot // PAGE, slot % PAGE
    h = torch.arange(H, device=x.device)[None, :, None, None]
    b16 = torch.arange(16, device=x.device)
    at = _seats(off)[:, None, :, None] + b16
    pool[blk[:, None, None, None], h, at] = by
    par = dz.reshape(n, H, 8).view(torch.uint8)
    pool[blk[:, None, None], h[..., 0], (CODES + 16 * off)[:, None, None] + b16] = par


def _values(codes, par):
    """codes uint8 [n, 4, 16] by group, par uint8 [n, 16] -> bf16 values [n, 128]."""
    n = codes.shape[0]
    by = codes.reshape(n, 4, 4, 2, 2).int()      # [n, g, w, e, i / 2]
    c = torch.stack([by & 15, by >> 4], -1)      # [n, g, w, e, i / 2, i % 2]
    c = c.permute(0, 1, 2, 4, 5, 3).reshape(n, 4, GROUP).float()
    dz = par.contiguous().view(torch.bfloat16).reshape(n, 4, 2).float()
    return (dz[..., 1:] + dz[..., :1] * (1.0 + c / 16.0)).bfloat16().reshape(n, DIM)


def _pages(pool, ids):
    """Pages ids [...] of a pool -> bf16 [..., H, 16, 128]."""
    page = pool[ids]
    H, n = pool.shape[1], ids.numel()
    code = page[..., :CODES].reshape(n * H, PAGE, 4, 16)
    t = torch.arange(PAGE, device=pool.device)
    g = torch.arange(4, device=pool.device)
    code = code[:, t[:, None], g[None, :] ^ ((t[:, None] >> 1) & 3)]
    v = _values(code.reshape(-1, 4, 16), page[..., CODES:].reshape(-1, 16))
    return v.reshape(*ids.shape, H, PAGE, DIM)


def _load(pool, slots):
    """Rows of the slots [n] -> bf16 [n, H, 128]; zeros for negative ones."""
    n, H = slots.shape[0], pool.shape[1]
    slot = slots.clamp(min=0)
    blk, off = slot // PAGE, slot % PAGE
    h = torch.arange(H, device=pool.device)[None, :, None, None]
    b16 = torch.arange(16, device=pool.device)
    code = pool[blk[:, None, None, None], h, _seats(off)[:, None, :, None] + b16]
    par = pool[blk[:, None, None], h[..., 0], (CODES + 16 * off)[:, None, None] + b16]
    v = _values(code.reshape(n * H, 4, 16), par.reshape(n * H, 16)).reshape(n, H, DIM)
    return torch.where((slots >= 0)[:, None, None], v, torch.zeros_like(v))


def _attend(s):
    """Causal softmax attention of every row, padded to the longest one."""
    k = _pages(s["k_cache"], s["tables"].clamp(min=0).long()).transpose(1, 2).flatten(2, 3).float()
    v = _pages(s["v_cache"], s["tables"].clamp(min=0).long()).transpose(1, 2).flatten(2, 3).float()
    R, H, T = k.shape[:3]
    indptr, lens = s["qo_indptr"].long(), s["seq_lens"].long()
    tok = torch.arange(s["q"].shape[0], device=k.device)
    r = torch.searchsorted(indptr, tok, right=True) - 1
    j = tok - indptr[r]
    n_q = int((s["qo_indptr_host"][1:] - s["qo_indptr_host"][:-1]).max())
    q = torch.zeros(R, n_q, H * QPK, DIM, device=k.device)
    q[r, j] = s["q"].float()
    q = q.reshape(R, n_q, H, QPK, DIM).permute(0, 2, 1, 3, 4).reshape(R, H, n_q * QPK, DIM)
    sc = (q @ k.transpose(-1, -2)).mul_(s["sm_scale"])
    last = lens - (indptr[1:] - indptr[:-1])     # position of a row's first query
    seen = torch.arange(T, device=k.device) <= (last[:, None] + torch.arange(n_q, device=k.device))[:, :, None]
    seen = seen & (torch.arange(T, device=k.device) < lens[:, None, None])
    seen = seen.repeat_interleave(QPK, 1)[:, None]
    sc.masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l
    lse = m + torch.log(l)
    o = o.reshape(R, H, n_q, QPK, DIM).transpose(1, 2).reshape(R, n_q, H * QPK, DIM)[r, j]
    lse = lse.reshape(R, H, n_q, QPK).transpose(1, 2).reshape(R, n_q, H * QPK)[r, j]
    return o.bfloat16(), lse


# ---------------------------------------------------------------------- cases
def _rows(gen, n, H, spread, device):
    """Keys or values [n, H, 128]: normal, each channel with a scale and an
    offset of its own (keys have such channels; spread 0: none)."""
    x = torch.randn(n, H, DIM, generator=gen, device=device)
    scale = torch.exp(spread * torch.randn(H, DIM, generator=gen, device=device))
    shift = spread * torch.randn(H, DIM, generator=gen, device=device)
    return (x * scale + shift).bfloat16()


def _lengths(case):
    """Tokens and queries of every row: the case's own, whatever the seed."""
    R = case["rows"]
    gen = torch.Generator().manual_seed(R * 1000003 + case["lo"] * 1009 + case["hi"])
    lens = torch.randint(case["lo"], case["hi"] + 1, (R,), generator=gen)
    n_q = torch.ones(R, dtype=torch.int64)
    many = R if case["q_rows"] == 0 else case["q_rows"]
    n_q[:many] = lens[:many] if case["q"] < 0 else torch.minimum(lens[:many], torch.tensor(case["q"]))
    if case["empty"]:
        n_q[case["empty"] - 1::case["empty"]] = 0
    return lens, n_q


def prepare(case, seed):
    """The pools with their cached tokens, the step's tensors and metadata on
    the device with host copies, and the buffers a serving loop keeps."""
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    H = case["kv_heads"]
    s = dict(op=case["op"])
    if case["op"] in ("write", "read"):
        n = case["tokens"]
        blocks = -(-n // PAGE) + 3
        slots = torch.randperm(blocks * PAGE, generator=host)[:n].to(dev)
        if case["op"] == "read" or n > 4096:     # long stretches lie in pages of one request each
            page = torch.randperm(blocks, generator=host)[:-(-n // PAGE)].to(dev)
            slots = (page[:, None] * PAGE + torch.arange(PAGE, device=dev)).flatten()[:n].contiguous()
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1
        cached = slots if case["op"] == "read" else None
        k, v = _rows(gen, n, H, 0.5, dev), _rows(gen, n, H, 0.0, dev)
        if case["op"] == "write":
            s.update(k_new=k, v_new=v)
        s.update(slots=slots, k_out=torch.empty_like(k), v_out=torch.empty_like(v))
    else:
        lens, n_q = _lengths(case)
        R, pages = case["rows"], (lens + PAGE - 1) // PAGE
        blocks = int(pages.sum()) + 3
        perm = torch.randperm(blocks, generator=host)
        first = torch.cumsum(pages, 0) - pages
        col = torch.arange(int(pages.max()))
        tables = torch.where(col < pages[:, None], perm[(first[:, None] + col).clamp(max=blocks - 1)], -1)
        indptr = torch.zeros(R + 1, dtype=torch.int64)
        indptr[1:] = torch.cumsum(n_q, 0)
        total = int(indptr[-1])
        row = torch.repeat_interleave(torch.arange(R), n_q)
        pos = (lens - n_q)[row] + torch.arange(total) - indptr[row]
        new = tables[row, pos // PAGE] * PAGE + pos % PAGE
        # every slot of the pages in use holds a token, the step's own ones excepted
        cached = (perm[:, None] * PAGE + torch.arange(PAGE)).flatten().to(dev)
        n = cached.shape[0]
        k, v = _rows(gen, n, H, 0.5, dev), _rows(gen, n, H, 0.0, dev)
        kn, vn = _rows(gen, total, H, 0.5, dev), _rows(gen, total, H, 0.0, dev)
        s.update(k_new=kn, v_new=vn, slots=new.to(dev), q=_rows(gen, total, H * QPK, 0.0, dev),
                 tables=tables.to(torch.int32).to(dev), seq_lens=lens.to(torch.int32).to(dev),
                 qo_indptr=indptr.to(torch.int32).to(dev), seq_lens_host=lens.to(torch.int32),
                 qo_indptr_host=indptr.to(torch.int32), sm_scale=1.0 / math.sqrt(DIM))
        s.update(out=torch.empty_like(s["q"]),
                 lse=torch.empty(total, H * QPK, dtype=torch.float32, device=dev))
    s["k_cache"] = torch.zeros(blocks, H, SLAB, dtype=torch.uint8, device=dev)
    s["v_cache"] = torch.zeros(blocks, H, SLAB, dtype=torch.uint8, device=dev)
    if cached is not None:
        _store(k, cached, s["k_cache"])
        _store(v, cached, s["v_cache"])
    if own:
        from paged_kv_decode_varlen_gb300 import binding as B
        s["binding"] = B
        size = B.PA_ERROR_WORD_BYTES
        if "q" in s:
            size = B.pa_attention_workspace_size(case["rows"], s["q"].shape[0], H * QPK, DIM, int(lens.max()))
        s["workspace"] = B.new_workspace(size, dev)
    return s


def run(s):
    if own:
        B, ws = s["binding"], s["workspace"]
        if s["op"] in ("write", "step"):
            B.pa_kv_append_q4(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"], workspace=ws)
        if s["op"] in ("write", "read"):
            return B.pa_kv_read_q4(s["slots"], s["k_cache"], s["v_cache"], k_out=s["k_out"], v_out=s["v_out"],
                                   workspace=ws)
        return B.pa_attention_varlen_q4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"],
                                        s["qo_indptr"], s["sm_scale"], seq_lens_host=s["seq_lens_host"],
                                        qo_indptr_host=s["qo_indptr_host"], out=s["out"], lse=s["lse"], workspace=ws)
    if s["op"] in ("write", "step"):
        _store(s["k_new"], s["slots"], s["k_cache"])
        _store(s["v_new"], s["slots"], s["v_cache"])
    if s["op"] in ("write", "read"):
        return _load(s["k_cache"], s["slots"]), _load(s["v_cache"], s["slots"])
    return _attend(s)


def work(case):
    """Bytes: each input once, each output once (a row's cached tokens are
    read once, whatever the number of its queries).  Flops: the two products."""
    H = case["kv_heads"]
    full, packed = 2 * H * DIM * 2, 2 * H * SLAB // PAGE    # a token's K and V as bf16, as 4-bit
    if case["op"] in ("write", "read"):
        n = case["tokens"]
        live = n - (n // case["skip"] if case["skip"] else 0)
        b = 8 * n + live * packed + n * full                # slots; codes read; rows written
        if case["op"] == "write":
            b += 8 * n + live * (full + packed)
        return {"bytes": b, "flops": 0}
    lens, n_q = _lengths(case)
    live = lens[n_q > 0]
    total = int(n_q.sum())
    pairs = int((n_q * (lens - n_q) + n_q * (n_q + 1) // 2).sum())
    b = int(live.sum()) * packed + int((-(-live // PAGE)).sum()) * 4
    b += total * H * QPK * (2 * DIM * 2 + 4) + 8 * case["rows"] + 4
    if case["op"] == "step":
        b += total * (full + packed + 8)
    return {"bytes": b, "flops": 4 * DIM * QPK * H * pairs}


# ------------------------------------------------------- the definition in 64 bits
def _exact_rows(x):
    """What rows x stand for once quantised: bf16 [n, H, 128] -> float64."""
    v = x.double().reshape(*x.shape[:-1], DIM // GROUP, GROUP)
    lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
    step = ((hi - lo) * 16 / 15).bfloat16().double()
    base = (lo - step).bfloat16().double()
    code = torch.floor(torch.clamp(16 * (v - base) / step - 16 + 0.5, 0, 15.5))
    # halves go to the even code
    tie = (16 * (v - base) / step - 16 + 0.5 == code) & (code % 2 == 1)
    code = torch.nan_to_num(torch.where(tie, code - 1, code))
    return (base + step * (16 + code) / 16).bfloat16().double().reshape(x.shape)


def _exact_slots(pool, slots):
    """The rows of slots [n] of a pool, float64 [n, H, 128]: every dim's bits
    looked up by their place."""
    dim = torch.arange(DIM, device=pool.device)
    g, w, e, i = dim // 32, dim % 32 // 8, dim % 2, dim % 8 // 2
    slab = pool[slots // PAGE]
    t = slots % PAGE
    place = 64 * t[:, None] + 16 * torch.bitwise_xor(g[None], (t[:, None] // 2) % 4) + 4 * w + 2 * e + i // 2
    n, H = slab.shape[:2]
    byte = torch.gather(slab, 2, place[:, None, :].expand(n, H, DIM)).double()
    code = torch.where(i % 2 == 1, torch.floor(byte / 16), byte % 16)
    at = CODES + 16 * t[:, None] + 4 * g[None]
    half = [torch.gather(slab, 2, (at + b)[:, None, :].expand(n, H, DIM)).int() for b in range(4)]
    D = ((half[0] << 16) | (half[1] << 24)).view(torch.float32).double()
    Z = ((half[2] << 16) | (half[3] << 24)).view(torch.float32).double()
    return (Z + D * (16 + code) / 16).bfloat16().double()


def exact(case, seed):
    s = prepare(case, seed)
    slots = s["slots"]
    if case["op"] == "write":
        keep = (slots >= 0)[:, None, None]
        return tuple(torch.where(keep, _exact_rows(x), 0.0) for x in (s["k_new"], s["v_new"]))
    if case["op"] == "read":
        keep = (slots >= 0)[:, None, None]
        return tuple(torch.where(keep, _exact_slots(s[c], slots.clamp(min=0)), 0.0) for c in ("k_cache", "v_cache"))
    outs, lses = [], []
    kn, vn = (_exact_rows(s["k_new"]), _exact_rows(s["v_new"])) if case["op"] == "step" else (None, None)
    H = case["kv_heads"]
    for r in range(case["rows"]):
        q0, q1, L = int(s["qo_indptr_host"][r]), int(s["qo_indptr_host"][r + 1]), int(s["seq_lens_host"][r])
        if q1 == q0:
            continue
        pos = torch.arange(L, device=slots.device)
        at = s["tables"][r].long()[pos // PAGE] * PAGE + pos % PAGE
        k, v = _exact_slots(s["k_cache"], at), _exact_slots(s["v_cache"], at)
        if kn is not None:
            k[L - (q1 - q0):], v[L - (q1 - q0):] = kn[q0:q1], vn[q0:q1]
        q = s["q"][q0:q1].double().reshape(q1 - q0, H, QPK, DIM)
        sc = torch.einsum("nhgd,thd->nhgt", q, k) * s["sm_scale"]
        late = pos > (L - (q1 - q0) + torch.arange(q1 - q0, device=slots.device))[:, None]
        sc = sc.masked_fill(late[:, None, None, :], -math.inf)
        outs.append(torch.einsum("nhgt,thd->nhgd", torch.softmax(sc, -1), v).reshape(q1 - q0, H * QPK, DIM))
        lses.append(torch.logsumexp(sc, -1).reshape(q1 - q0, H * QPK))
    return torch.cat(outs), torch.cat(lses)
