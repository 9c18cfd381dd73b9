"""q4 calls on a stream that is not the current one, and from several host
threads at once."""
import threading

import pytest
import torch

from tests.test_gpu_q4 import Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B


def test_lengths_written_on_the_calls_stream_are_read_there():
    """Without host copies the lengths are fetched behind the stream's work,
    which here writes them late."""
    c = Case([300, 45, 700], [1, 9, 4], 2, seed=5)
    want, want_lse = c.run()
    d = c.dev
    seq, ind = torch.ones_like(d["seq"]), torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    pinned = [torch.empty(t.shape, dtype=t.dtype, pin_memory=True).copy_(t) for t in (d["seq"], d["ind"])]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # some 50 ms
        seq.copy_(pinned[0], non_blocking=True)
        ind.copy_(pinned[1], non_blocking=True)
    out, lse = B.pa_attention_varlen_q4(d["q"], c.kc, c.vc, d["tables"], seq, ind, c.b.sm_scale, stream=side,
                                        return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_threads_call_at_once():
    cases = [Case([1200, 300, 50], [1, 30, 5], 2, seed=41 + i) for i in range(4)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * len(cases), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [cases[i].run() for _ in range(40)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # shown below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for (out, lse), runs in zip(want, got):
        assert all(torch.equal(o, out) and torch.equal(x, lse) for o, x in runs)
