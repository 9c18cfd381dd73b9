"""pa_step_tables through the C ABI: every output equals the oracle's, which
walks requests, tokens and pages one at a time."""
import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

DEV = "cuda"
KEYS = ("seq_lens", "qo_indptr", "slot_mapping", "positions", "free_state", "first_page", "block_tables", "free_ring")


def make(R, cached, new, window=0, sinks=0, shared=0, spare=4, max_blocks=None, pad=3, seed=0, gone=True):
    """A step of R requests: tables that hold what the step before left, the
    other blocks in the ring."""
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached, np.int64), np.asarray(new, np.int64)
    had, has = -(-cached // 16), -(-(cached + np.maximum(new, 0)) // 16)
    keep = max(-(-sinks // 16) if window else 0, shared)
    first = np.zeros(R, np.int64)
    if window and gone:
        upto = np.maximum(cached - window, 0) // 16
        first = np.where(upto > keep, upto, 0)
    mb = max_blocks or max(1, int(has.max(initial=1)) + 1)
    tables = np.full((R, mb), -1, np.int32)
    held = [(r, j) for r in range(R) for j in range(min(int(had[r]), mb)) if j < keep or j >= first[r]]
    nb = len(held) + int((has - had).sum()) + spare
    perm = rng.permutation(nb).astype(np.int32)
    for i, (r, j) in enumerate(held):
        tables[r, j] = perm[i]
    free = perm[len(held):]
    head = int(rng.integers(0, nb))
    ring = np.full(nb, -1, np.int32)
    ring[(head + np.arange(len(free))) % nb] = free
    total = int(np.maximum(new, 0).sum())
    return dict(new=new.astype(np.int32), cached=cached.astype(np.int32), first=first.astype(np.int32), tables=tables,
                ring=ring, state=np.array([head, len(free)], np.int32), window=window, sinks=sinks, shared=shared,
                n_tokens=total + pad)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run(c, **kw):
    tables, ring = dev(c["tables"]), dev(c["ring"])
    ws = kw.pop("workspace", None)
    ws = B.new_workspace(256, DEV) if ws is None else ws
    out = B.pa_step_tables(dev(c["new"]), dev(c["cached"]), tables, ring, dev(c["state"]), n_tokens=c["n_tokens"],
                           window=c["window"], sink_tokens=c["sinks"], shared_pages=c["shared"], first_page=dev(c["first"]),
                           workspace=ws, **kw)
    torch.cuda.synchronize()
    got = dict(zip(KEYS, out))
    got.update(block_tables=tables, free_ring=ring)
    assert not ws[4:].any()  # nothing but the error word is left
    return {k: v.cpu().numpy() for k, v in got.items()}, B.pa_get_device_error(ws)


def check(c, **kw):
    got, err = run(c, **kw)
    want, errors = step.step_tables(c["new"], c["cached"], c["first"], c["tables"], c["ring"], c["state"], c["window"],
                                    c["sinks"], c["shared"], c["n_tokens"])
    for k in KEYS:
        assert np.array_equal(got[k], want[k]), (k, np.argwhere(got[k] != want[k])[:5].tolist())
    assert (err in errors) if errors else err == 0
    return want


def lens(seed, R, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi + 1, R)


CASES = {
    "one": dict(R=1, cached=[0], new=[1]),
    "page_edges": dict(R=8, cached=[0, 15, 16, 17, 31, 32, 33, 48], new=[1, 1, 1, 1, 2, 16, 15, 17]),
    "decode": dict(R=64, cached=lens(1, 64, 0, 5000), new=[1] * 64),
    "nobody": dict(R=5, cached=[3, 0, 16, 17, 100], new=[0] * 5),
    "no_requests": dict(R=0, cached=[], new=[]),
    "ended": dict(R=7, cached=[100, 0, 16, 1, 500, 64, 15], new=[-1, -1, -7, 3, -1, 20, -2]),
    "windows": dict(R=40, cached=lens(2, 40, 0, 900), new=lens(3, 40, -1, 40), window=100, sinks=4),
    "window_of_one": dict(R=20, cached=lens(4, 20, 0, 100), new=lens(5, 20, -1, 3), window=1),
    "first_release": dict(R=12, cached=lens(6, 12, 0, 2000), new=lens(7, 12, 0, 2), window=300, sinks=33, gone=False),
    "shared_prefix": dict(R=9, cached=lens(8, 9, 48, 700), new=lens(9, 9, -1, 30), window=64, sinks=4, shared=3),
    "shared_no_window": dict(R=9, cached=lens(10, 9, 48, 700), new=lens(11, 9, -1, 30), sinks=4, shared=3),
    "chunks": dict(R=5, cached=[0, 700, 3, 0, 129], new=[3000, 1, 1500, 0, 777], window=512),
    "rows_over_a_block": dict(R=2600, cached=lens(12, 2600, 0, 200), new=lens(13, 2600, -1, 5), window=50, sinks=1),
    "many_rows": dict(R=20000, cached=lens(14, 20000, 0, 60), new=lens(15, 20000, -1, 2), window=20),
    "wide_window": dict(R=4, cached=[1000, 5, 70, 900], new=[1, -1, 3, 40], window=2 ** 31 - 1, sinks=2 ** 31 - 1),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_equals_the_oracle(name):
    check(make(**CASES[name], seed=len(name)))


def test_no_padding_and_much_of_it():
    for pad in (0, 5000):
        check(make(9, lens(1, 9, 0, 300), lens(2, 9, 0, 50), pad=pad))


@pytest.mark.parametrize("left", [0, 1, 5])
def test_the_ring_runs_out(left):
    c = make(6, [16, 0, 33, 5, 48, 100], [1, 40, 1, 60, 1, -1], seed=left)
    c["state"][1] = left
    got = check(c)
    assert (got["slot_mapping"][:103] < 0).any() and got["free_state"][1] == 7  # what the ended request held


def test_rows_out_of_bounds_wait():
    c = make(8, [10, 20, 30, 40, 50, 60, 70, 80], [1, 1, 1, 1, 1, 1, 1, -1], max_blocks=6)
    c["cached"][1], c["cached"][2], c["new"][3], c["cached"][5] = -5, 97, 57, (1 << 20) + 1
    got = check(c)
    assert got["seq_lens"].tolist() == [11, 0, 0, 40, 51, 0, 71, 0]


def test_too_many_tokens_or_a_broken_ring_change_nothing():
    base = make(5, [10, 20, 30, 40, 50], [1, 40, 1, 1, -1], pad=0)
    for change in (dict(n_tokens=42), dict(state=np.array([-1, 3], np.int32)), dict(state=np.array([0, -1], np.int32)),
                   dict(state=np.array([len(base["ring"]), 3], np.int32)), dict(state=np.array([0, len(base["ring"]) + 1], np.int32)),
                   # the ended request's four pages do not fit behind what the ring says it has
                   dict(state=np.array([0, len(base["ring"])], np.int32))):
        c = dict(base, **change)
        got = check(c)
        assert np.array_equal(got["block_tables"], c["tables"]) and np.array_equal(got["free_ring"], c["ring"])
        assert np.array_equal(got["free_state"], c["state"]) and got["qo_indptr"][-1] == 0


def test_ids_outside_the_pool_are_granted_as_none():
    c = make(4, [16, 32, 48, 64], [1, 1, 1, 1], seed=3)
    at = (c["state"][0] + np.arange(4)) % len(c["ring"])
    c["ring"][at[1]], c["ring"][at[2]] = len(c["ring"]), -7
    got = check(c)
    assert (got["slot_mapping"][:4] < 0).tolist() == [False, True, True, False]


def test_a_large_sum_of_new_tokens_does_not_wrap():
    # 4096 rows of 2^20 tokens: 2^32 in all
    c = make(4096, [0] * 4096, [0] * 4096, max_blocks=1 << 16, spare=10)
    c["new"][:] = 1 << 20
    check(c)


def test_optional_arrays_may_be_left_out():
    c = make(3, [5, 16, 40], [1, 1, -1])
    want, _ = step.step_tables(c["new"], c["cached"], c["first"], c["tables"], c["ring"], c["state"], 0, 0, 0, 2)
    tables, ring = dev(c["tables"]), dev(c["ring"])
    out = B.pa_step_tables(dev(c["new"]), dev(c["cached"]), tables, ring, dev(c["state"]), n_tokens=2)
    for got, k in zip(out, KEYS):
        assert np.array_equal(got.cpu().numpy(), want[k]), k


def test_a_captured_call_steps_on_in_place():
    """Lengths, ring state and first pages updated in place: every replay is
    the next step; requests end and new ones take their rows in between."""
    c = make(70, lens(20, 70, 0, 400), [1] * 70, window=64, sinks=4, spare=300, max_blocks=60, pad=10)
    t = {k: dev(c[k]) for k in ("new", "cached", "first", "tables", "ring", "state")}
    ws = B.new_workspace(256, DEV)
    out = dict(qo_indptr=torch.empty(71, dtype=torch.int32, device=DEV), slot_mapping=torch.empty(80, dtype=torch.int64, device=DEV),
               positions=torch.empty(80, dtype=torch.int32, device=DEV))

    def call():
        B.pa_step_tables(t["new"], t["cached"], t["tables"], t["ring"], t["state"], window=64, sink_tokens=4,
                         first_page=t["first"], seq_lens=t["cached"], free_state_out=t["state"], first_page_out=t["first"],
                         workspace=ws, **out)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    rng = np.random.default_rng(21)
    h = {k: c[k].copy() for k in t}
    for i in range(40):
        h["new"] = np.where(h["cached"] == 0, rng.integers(0, 2, 70), np.where(rng.random(70) < 0.05, -1, 1)).astype(np.int32)
        t["new"].copy_(torch.from_numpy(h["new"]))
        graph.replay()
        want, errors = step.step_tables(h["new"], h["cached"], h["first"], h["tables"], h["ring"], h["state"], 64, 4, 0, 80)
        assert not errors
        h.update(cached=want["seq_lens"], first=want["first_page"], state=want["free_state"], tables=want["block_tables"],
                 ring=want["free_ring"])
        torch.cuda.synchronize()
        for k in ("cached", "first", "state", "tables", "ring"):
            assert np.array_equal(t[k].cpu().numpy(), h[k]), (i, k)
        for k in out:
            assert np.array_equal(out[k].cpu().numpy(), want[k]), (i, k)
    assert B.pa_get_device_error(ws) == 0


def test_in_place_with_many_blocks_of_threads():
    c = make(3000, lens(22, 3000, 0, 90), lens(23, 3000, -1, 3), window=40, pad=9000)
    want = check(c)
    cached, state, first = dev(c["cached"]), dev(c["state"]), dev(c["first"])
    tables, ring = dev(c["tables"]), dev(c["ring"])
    B.pa_step_tables(dev(c["new"]), cached, tables, ring, state, n_tokens=c["n_tokens"], window=40, first_page=first,
                     seq_lens=cached, free_state_out=state, first_page_out=first)
    for got, k in ((cached, "seq_lens"), (state, "free_state"), (first, "first_page"), (tables, "block_tables"), (ring, "free_ring")):
        assert np.array_equal(got.cpu().numpy(), want[k]), k


def test_on_a_stream_that_is_not_the_current_one():
    c = make(30, lens(24, 30, 0, 300), lens(25, 30, -1, 30), window=80, sinks=4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    check(c, stream=side)
