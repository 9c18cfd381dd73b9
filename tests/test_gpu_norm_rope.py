"""pa_qk_norm_rope and pa_qk_norm_rope_append through the C ABI against the
formula in 64 bits.

Bounds.  A result is rounded once to bf16: 2^-8 of it.  Before that, in binary32:
the mean of 128 squares and its root (some 25 roundings of 2^-24, halved by the
root), the weight and the pair's two products (4 more): 2^-19 of |a| + |b|.  The
angle is the upper 32 bits of a 64-bit fraction of a turn (2^-32 turns) rounded to
binary32 (2^-24 of half a turn at most), of a speed off by 2^-52 relative and
2^-64 turns per position (up to 2^20): below 2^-21 radians in all; sine and cosine
are within 2 units in the last place, 2^-22: together 2^-20 of |a| + |b|.
  |out - ref| <= 2^-8 |ref| + 2^-18 (|a| + |b|).
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


def speeds(rotary, base=1e6):
    return base ** (-np.arange(0, rotary, 2) / rotary)


class Case:
    def __init__(self, N, Hkv, rotary=128, inter=False, norm=True, fused=False, far=5000, seed=0, kind="normal", eps=1e-6):
        rng = np.random.default_rng(seed)
        self.N, self.Hkv, self.inter, self.eps = N, Hkv, inter, eps
        H = 6 * Hkv
        x = rng.standard_normal((N, H, 128)).astype(np.float32)
        if kind == "spread":
            x *= np.exp2(rng.integers(-20, 21, (N, H, 1))).astype(np.float32)
        elif kind == "tiny":
            x *= np.float32(2.0 ** -60)
        elif kind == "zero":
            x[:, ::2] = 0
        self.x = W.f32_to_bf16_bits(x)
        self.q, self.k, self.v = self.x[:, :4 * Hkv], self.x[:, 4 * Hkv:5 * Hkv], self.x[:, 5 * Hkv:]
        self.pos = rng.integers(0, far, N).astype(np.int32)
        if N:
            self.pos[0], self.pos[-1] = 0, far - 1
        self.f = speeds(rotary)
        self.qw, self.kw = ((1 + 0.3 * rng.standard_normal(128)).astype(np.float32) if norm else None for _ in range(2))
        if fused:
            wide = bf16_dev(self.x)
            self.dq, self.dk, self.dv = wide[:, :4 * Hkv], wide[:, 4 * Hkv:5 * Hkv], wide[:, 5 * Hkv:]
        else:
            self.dq, self.dk, self.dv = bf16_dev(self.q), bf16_dev(self.k), bf16_dev(self.v)
        self.kw_args = dict(q_weight=None if self.qw is None else torch.from_numpy(self.qw).to(DEV),
                            k_weight=None if self.kw is None else torch.from_numpy(self.kw).to(DEV), eps=eps, interleaved=inter)
        self.dpos = torch.from_numpy(self.pos).to(DEV)
        self.turns = B.pa_rope_turns(self.f).to(DEV)

    def near(self, got, x, w, what):
        ref, size = step.norm_rope(x, w, self.pos, self.f, self.eps, self.inter)
        err = np.abs(oracle.bf16_to_f64(got) - ref)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * size
        bad = ~(err <= tol)
        assert not bad.any(), (what, np.argwhere(bad)[:5].tolist(), float(np.nanmax(err / np.maximum(tol, 1e-300))))

    def plain(self, **kw):
        return B.pa_qk_norm_rope(self.dq, self.dk, self.dpos, self.turns, **self.kw_args, **kw)

    def append(self, slots, kc, vc, **kw):
        return B.pa_qk_norm_rope_append(self.dq, self.dk, self.dv, self.dpos, torch.from_numpy(slots).to(DEV), self.turns,
                                        kc, vc, **self.kw_args, **kw)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 32, 48, 64, 96, 112, 128])
def test_rotary_dims(rotary, inter):
    c = Case(11, 2, rotary, inter, seed=rotary)
    q, k = c.plain()
    c.near(bf16_host(q), c.q, c.qw, "q")
    c.near(bf16_host(k), c.k, c.kw, "k")


@pytest.mark.parametrize("N,Hkv", [(1, 1), (1, 8), (3, 1), (2, 3), (64, 8), (33, 2), (500, 1), (7, 5), (3, 40), (1201, 2)])
@pytest.mark.parametrize("fused", [False, True])
def test_sizes_and_strides(N, Hkv, fused):
    c = Case(N, Hkv, fused=fused, seed=N)
    q, k = c.plain()
    c.near(bf16_host(q), c.q, c.qw, "q")
    c.near(bf16_host(k), c.k, c.kw, "k")


@pytest.mark.parametrize("kind", ["spread", "tiny", "zero"])
@pytest.mark.parametrize("norm", [False, True])
def test_values(kind, norm):
    c = Case(20, 2, norm=norm, kind=kind)
    q, k = c.plain()
    c.near(bf16_host(q), c.q, c.qw, "q")
    c.near(bf16_host(k), c.k, c.kw, "k")


@pytest.mark.parametrize("base", [1e4, 1e9])
def test_far_positions(base):
    c = Case(300, 1, far=1 << 20, seed=4)
    c.f = speeds(128, base)
    c.turns = B.pa_rope_turns(c.f).to(DEV)
    q, k = c.plain()
    c.near(bf16_host(q), c.q, c.qw, "q")


def test_negative_positions_turn_backwards():
    c = Case(16, 1, seed=5)
    c.pos = -c.pos
    c.dpos = -c.dpos
    q, _ = c.plain()
    c.near(bf16_host(q), c.q, c.qw, "q")


def test_the_norm_of_q_alone():
    c = Case(9, 2, seed=6)
    c.kw = c.kw_args["k_weight"] = None
    q, k = c.plain()
    c.near(bf16_host(q), c.q, c.qw, "q")
    c.near(bf16_host(k), c.k, None, "k")


def test_in_place():
    c = Case(40, 3, seed=7)
    want_q, want_k = c.plain()
    q, k = c.plain(q_out=c.dq, k_out=c.dk)
    assert q is c.dq and torch.equal(q, want_q) and torch.equal(k, want_k)


def test_not_a_number_stays_in_its_row():
    c = Case(6, 2, seed=8)
    want, _ = c.plain()
    c.dq[2, 3, 5], c.dq[4, 0, 100] = float("nan"), float("inf")
    got, _ = c.plain()
    assert bool(torch.isnan(got[2, 3]).all()) and bool(torch.isnan(got[4, 0, 100]))
    keep = torch.ones(6, 8, dtype=torch.bool, device=DEV)
    keep[2, 3] = keep[4, 0] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("N,Hkv,fused", [(1, 8, True), (64, 8, True), (37, 1, False), (50, 2, True), (5, 20, False), (900, 5, True)])
def test_append(N, Hkv, fused):
    c = Case(N, Hkv, fused=fused, seed=N + 1)
    rng = np.random.default_rng(N)
    nb = N // 16 + 3
    slots = rng.permutation(nb * 16)[:N].astype(np.int64)
    slots[3::5] = -1
    kc = bf16_dev(rng.integers(0, 1 << 16, (nb, Hkv, 16, 128)).astype(np.uint16))
    vc = bf16_dev(rng.integers(0, 1 << 16, (nb, Hkv, 16, 128)).astype(np.uint16))
    hk, hv = bf16_host(kc).copy(), bf16_host(vc).copy()
    ws = B.new_workspace(256, DEV)
    q = c.append(slots, kc, vc, workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == 0
    c.near(bf16_host(q), c.q, c.qw, "q")
    _, want_k = c.plain()
    live = slots >= 0
    hk[slots[live] // 16, :, slots[live] % 16] = bf16_host(want_k)[live]   # held to the formula above
    hv[slots[live] // 16, :, slots[live] % 16] = c.v[live]
    assert np.array_equal(bf16_host(kc), hk) and np.array_equal(bf16_host(vc), hv)


def test_append_records_bad_slots_and_leaves_the_rest():
    c = Case(4, 2, seed=9)
    kc = torch.full((3, 2, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    ws = B.new_workspace(256, DEV)
    q = c.append(np.array([48, 17, 1 << 50, -1 << 40]), kc, vc, workspace=ws)
    torch.cuda.synchronize()
    assert B.pa_get_device_error(ws) == B.PA_ERR_DEVICE_INDEX
    c.near(bf16_host(q), c.q, c.qw, "q")
    assert torch.equal(vc[1, :, 1], c.dv[1])
    kc[1, :, 1] = vc[1, :, 1] = 7.0
    assert bool((kc == 7.0).all()) and bool((vc == 7.0).all())


def test_a_captured_call_takes_new_contents():
    c = Case(30, 2, seed=10)
    kc = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    vc, slots = torch.zeros_like(kc), torch.arange(30, device=DEV)
    q, ws = torch.empty_like(c.dq), B.new_workspace(256, DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.pa_qk_norm_rope_append(c.dq, c.dk, c.dv, c.dpos, slots, c.turns, kc, vc, q_out=q, workspace=ws, **c.kw_args)
    for i in range(3):
        d = Case(30, 2, seed=20 + i)
        for a, b in ((c.dq, d.dq), (c.dk, d.dk), (c.dv, d.dv), (c.dpos, d.dpos), (slots, slots.flip(0).clone())):
            a.copy_(b)
        for name in ("q_weight", "k_weight"):
            c.kw_args[name].copy_(d.kw_args[name])
        graph.replay()
        torch.cuda.synchronize()
        want_q, want_k = d.plain()
        assert torch.equal(q, want_q)
        assert torch.equal(kc[slots // 16, :, slots % 16], want_k) and torch.equal(vc[slots // 16, :, slots % 16], d.dv)


def test_on_a_stream_that_is_not_the_current_one():
    c = Case(100, 8, fused=True, seed=11)
    want = c.plain()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.plain(stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
