"""One workspace that serves attention with a window for batches of several
sizes, eager and captured, after calls of other kinds and whatever it held."""
import numpy as np
import pytest
import torch

from tests.test_gpu_window import DEV, Case, rand

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

# batches of 8, 2 and 3 kv heads; rows of one query, of several, prompt chunks; all with rows
# that are cut between CTAs
SIZES = [
    dict(seq=[3000, 2500, 4000], qo=[1] * 3, window=2000, sinks=4, Hkv=8),
    dict(seq=rand(3, 64, 300, 3000), qo=[1] * 64, window=900, sinks=4, Hkv=8),
    dict(seq=rand(4, 64, 300, 3000), qo=[1] * 64, window=900, sinks=0, Hkv=2),
    dict(seq=[5000], qo=[5], window=4000, sinks=4, Hkv=3),
    dict(seq=rand(5, 200, 900, 1500), qo=[1 + i % 6 for i in range(200)], window=700, sinks=4, Hkv=2),
    dict(seq=[3000, 40, 900, 2000], qo=[100, 1, 5, 1], window=1500, sinks=17, Hkv=8),
    dict(seq=rand(6, 300, 1, 140), qo=[1] * 300, window=100, sinks=4, Hkv=3),
]


def make():
    return [Case(**s, seed=60 + i) for i, s in enumerate(SIZES)]


def need(cases):
    return max(B.pa_window_workspace_size(len(c.seq), len(c.q), 4 * c.Hkv, 128, c.window, c.sinks) for c in cases)


def poison(want):
    """Outputs that a call has to write: of its results' shapes, and none of
    their values."""
    return torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)


def same(c, want, ws, call, what):
    out, lse = poison(want)
    call(out=out, lse=lse, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), what


def calls(c):
    return [c.run, c.decode] if max(c.qo) == 1 and min(c.qo) == 1 else [c.run]


def test_batches_of_several_sizes_share_a_workspace():
    cases = make()
    want = [[call() for call in calls(c)] for c in cases]
    for c, w in zip(cases, want):
        c.check(*w[0])
    ws = B.new_workspace(need(cases), DEV)
    n = len(cases)
    for order in (range(n), reversed(range(n)), [0, 1, 0, 1, 2, 1, 0, 4, 3, 4, 6, 5, 1]):
        for i in order:
            for call, w in zip(calls(cases[i]), want[i]):
                same(cases[i], w, ws, call, i)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


@pytest.mark.parametrize("fill", ["random", 0xff, 1])
def test_results_do_not_depend_on_what_the_workspace_held(fill):
    cases = make()
    want = [[call() for call in calls(c)] for c in cases]
    size = need(cases)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(8)
    for i in range(len(cases)):
        ws.copy_(torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV, generator=g)) if fill == "random" else ws.fill_(fill)
        ws[:B.PA_ERROR_WORD_BYTES] = 0
        for call, w in zip(calls(cases[i]), want[i]):
            same(cases[i], w, ws, call, i)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0


@pytest.mark.parametrize("Hkv", [2, 8])
def test_graphs_of_several_padded_sizes_share_a_workspace(Hkv):
    """Captured for 4, 16 and 64 rows and replayed in turn, each several times
    in a row, with other lengths every time."""
    window, sinks = 800, 4
    made = []
    biggest = Case([2000] * 64, [1] * 64, window, sinks, Hkv, seed=70)
    nb = biggest.k.shape[0]
    ws = biggest.workspace()
    for R in (4, 16, 64):
        t = dict(q=torch.zeros(R, 4 * Hkv, 128, dtype=torch.bfloat16, device=DEV), seq=torch.zeros(R, dtype=torch.int32, device=DEV),
                 tables=torch.full((R, 130), -1, dtype=torch.int32, device=DEV))
        for x in ("k", "v"):
            t[x] = torch.zeros(nb, Hkv, 16, 128, dtype=torch.bfloat16, device=DEV)
        out, lse = torch.empty_like(t["q"]), torch.empty(R, 4 * Hkv, device=DEV)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            B.pa_decode_window(t["q"], t["k"], t["v"], t["tables"], t["seq"], biggest.scale, window, sinks, out=out, lse=lse,
                               workspace=ws)
        made.append((R, t, out, lse, graph))
    for i, at in enumerate([0, 1, 2, 0, 0, 2, 1, 2, 2, 0, 1]):
        R, t, out, lse, graph = made[at]
        c = Case(rand(80 + i, R, 1, 2000), [1] * R, window, sinks, Hkv, seed=90 + i)
        t["tables"][:, :c.tables.shape[1]].copy_(c.d["tables"])
        for x in ("k", "v"):
            t[x][:c.k.shape[0]].copy_(c.d[x])
        t["q"].copy_(c.d["q"])
        t["seq"].copy_(c.d["seq"])
        out.fill_(7.0)
        lse.fill_(7.0)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse, what=f"replay {i}, {R} rows")
    assert B.pa_get_device_error(ws) == 0


def test_layers_with_and_without_a_window_share_a_workspace():
    """One batch, one workspace, calls in turn: neither finds the counts of the
    other's rows in its place."""
    for R, Hkv in ((20, 8), (3, 2), (130, 2)):
        seq = rand(R, R, 800, 2000)
        c = Case(seq, [1] * R, max(seq), 0, Hkv, seed=R)          # every key has its page
        c.window = 600
        d, host = c.d, dict(seq_lens_host=torch.from_numpy(c.seq), qo_indptr_host=torch.from_numpy(c.ind))
        size = max(c.workspace().numel(), B.pa_attention_workspace_size(R, R, 4 * Hkv, 128, max(seq)))
        ws = B.new_workspace(size, DEV)

        def plain(**kw):
            return B.pa_attention_varlen(d["q"], d["k"], d["v"], d["tables"], d["seq"], d["ind"], c.scale, return_lse=True,
                                         **host, **kw)

        want, narrow = plain(), c.run()
        for _ in range(3):
            same(c, want, ws, plain, "plain")
            same(c, narrow, ws, c.run, "window")
            same(c, narrow, ws, c.decode, "window, planned on the device")
        torch.cuda.synchronize()
        assert B.pa_get_device_error(ws) == 0


def test_the_size_does_not_shrink_with_a_larger_batch():
    last = 0
    for rows, total, heads in ((0, 0, 4), (1, 1, 4), (1, 6, 4), (1, 7, 4), (3, 64, 32), (64, 64, 32), (64, 4096, 32),
                               (65535, 65535, 32), (65535, 1 << 20, 1024)):
        size = B.pa_window_workspace_size(rows, total, heads, 128, 64, 4)
        assert size >= last, (rows, total, heads)
        last = size
