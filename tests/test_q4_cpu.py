"""q4 pages without a GPU: the format's oracle against what the format fixes,
and the refusals of the q4 calls (no call here reaches a kernel)."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import q4
from paged_kv_decode_varlen_gb300 import binding as b
from paged_kv_decode_varlen_gb300 import workloads as W

lib = b._lib
FAKE = ctypes.c_void_p(1 << 20)  # non-null, aligned; never dereferenced on these paths
ODD = ctypes.c_void_p((1 << 20) + 8)


def test_every_code_has_a_place_of_its_own():
    seen = set()
    for t in range(16):
        byte, shift = q4.places(t)
        assert set(byte // 64) == {t}
        seen |= set(zip(byte.tolist(), shift.tolist()))
    assert len(seen) == 16 * 128 and {s for _, s in seen} == {0, 4}
    # the documented word order: dims 0 and 1 of a group at bits 0 and 16
    byte, shift = q4.places(0)
    assert (byte[0], shift[0], byte[1], shift[1], byte[2], shift[2], byte[8], byte[32]) == (0, 0, 2, 0, 0, 4, 4, 16)
    assert q4.places(2)[0][0] == 2 * 64 + 16 and q4.places(15)[0][0] == 15 * 64 + 48


def test_rounding_to_bf16_keeps_subnormals():
    # ties to even at a normal, a subnormal and the smallest step (2^-133)
    x = np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 3 * 2.0 ** -134, 2.0 ** -134, -5 * 2.0 ** -133, 0.0, -0.0])
    assert q4.round_bf16(x).tolist() == [0x3f80, 0x3f82, 2, 0, 0x8005, 0, 0x8000]
    assert q4.round_bf16(np.array([np.nan, np.inf, -4e38, 3.3895e38])).tolist() == [0x7fc0, 0x7f80, 0xff80, 0x7f7f]
    rng = np.random.default_rng(1)
    y = rng.standard_normal(4096) * np.exp2(rng.integers(-120, 120, 4096))
    assert np.array_equal(q4.round_bf16(y), oracle.round_bf16(y))


def test_slab_constants_agree():
    assert b.PA_Q4_SLAB_BYTES == q4.SLAB == 1280


def _value(bits):
    return oracle.bf16_to_f64(bits)


def test_quantisation_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = W.normal_bf16(rng, (40, 2, 128))
    pool = np.zeros((5, 2, q4.SLAB), np.uint8)
    slots = rng.permutation(80)[:40].astype(np.int64)
    q4.append(x, slots, pool)
    got = _value(q4.unpack(pool))[slots // 16, :, slots % 16]
    v = _value(x)
    g = v.reshape(40, 2, 4, 32)
    span = g.max(-1) - g.min(-1)
    # half a step of a sixteenth of D inside the grid; D is span x 16/15 to
    # 2^-8, Z to 2^-8 of |lo| + D (so the grid's ends move by that much, and
    # at the top by 15/16 of D's rounding too), the value rounded to bf16
    d = span * 16 / 15 * (1 + 2.0 ** -8)
    bound = d / 32 + 2.0 ** -8 * (np.abs(g.min(-1)) + 2 * d) + 2.0 ** -8 * np.abs(g).max(-1)
    assert np.all(np.abs(got - v).reshape(40, 2, 4, 32) <= bound[..., None])


def test_the_largest_inputs_are_within_half_a_step():
    rng = np.random.default_rng(5)
    x = np.clip(rng.standard_normal((60, 1, 128)) * 2.0 ** 124.5, -2.0 ** 125, 2.0 ** 125).astype(np.float32)
    bits = W.f32_to_bf16_bits(x)
    pool = np.zeros((4, 1, q4.SLAB), np.uint8)
    q4.append(bits, np.arange(60), pool)
    got = _value(q4.unpack(pool))[np.arange(60) // 16, :, np.arange(60) % 16].reshape(60, 4, 32)
    v = _value(bits).reshape(60, 4, 32)
    # the bound of the test above
    d = (v.max(-1) - v.min(-1)) * 16 / 15 * (1 + 2.0 ** -8)
    bound = d / 32 + 2.0 ** -8 * (np.abs(v.min(-1)) + 2 * d) + 2.0 ** -8 * np.abs(v).max(-1)
    assert np.all(np.abs(got - v) <= bound[..., None])


def test_equal_values_are_exact_and_codes_span_the_range():
    x = np.full((1, 1, 128), 0x4049, np.uint16)
    pool = np.zeros((1, 1, q4.SLAB), np.uint8)
    q4.append(x, np.array([5]), pool)
    assert np.array_equal(q4.unpack(pool)[0, 0, 5], x[0, 0])
    ramp = W.f32_to_bf16_bits(np.tile(np.arange(32, dtype=np.float32) - 7, 4))
    codes, _, _ = q4.quantize(ramp[None, None])
    assert codes.min() == 0 and codes.max() == 15


def _append(**kw):
    a = dict(k=FAKE, v=FAKE, s=FAKE, n=4, kc=FAKE, vc=FAKE, nb=64, P=16, H=8, D=128, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.pa_kv_append_q4(a["k"], a["v"], a["s"], a["n"], a["kc"], a["vc"], a["nb"], a["P"], a["H"], a["D"],
                               a["ws"], a["wsb"], None)


def _read(**kw):
    a = dict(k=FAKE, v=FAKE, s=FAKE, n=4, kc=FAKE, vc=FAKE, nb=64, P=16, H=8, D=128, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.pa_kv_read_q4(a["s"], a["n"], a["kc"], a["vc"], a["nb"], a["P"], a["H"], a["D"], a["k"], a["v"],
                             a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [_append, _read], ids=["append", "read"])
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), b.PA_ERR_INVALID_ARG),
    (dict(nb=0), b.PA_ERR_INVALID_ARG),
    (dict(H=0), b.PA_ERR_INVALID_ARG),
    (dict(k=None), b.PA_ERR_INVALID_ARG),
    (dict(v=None), b.PA_ERR_INVALID_ARG),
    (dict(s=None), b.PA_ERR_INVALID_ARG),
    (dict(kc=None), b.PA_ERR_INVALID_ARG),
    (dict(ws=None), b.PA_ERR_INVALID_ARG),
    (dict(k=ODD), b.PA_ERR_INVALID_ARG),
    (dict(vc=ODD), b.PA_ERR_INVALID_ARG),
    (dict(s=ctypes.c_void_p((1 << 20) + 4)), b.PA_ERR_INVALID_ARG),
    (dict(D=64), b.PA_ERR_UNSUPPORTED),
    (dict(P=32), b.PA_ERR_UNSUPPORTED),
    (dict(H=257), b.PA_ERR_UNSUPPORTED),
    (dict(wsb=255), b.PA_ERR_WORKSPACE_TOO_SMALL),
    (dict(n=1 << 28), b.PA_ERR_UNSUPPORTED),   # 2^31 rows
])
def test_write_and_read_refusals(call, kw, status):
    n0 = lib.pa_launch_count()
    assert call(**kw) == status, lib.pa_last_error_message().decode()
    assert lib.pa_last_error_message().decode() != "" and lib.pa_launch_count() == n0


@pytest.mark.parametrize("call", [_append, _read], ids=["append", "read"])
def test_no_tokens_launch_nothing(call):
    n0 = lib.pa_launch_count()
    assert call(n=0, k=None, v=None, s=None) == b.PA_OK and lib.pa_launch_count() == n0


def _attn(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, nb=64, bt=FAKE, mb=40, sl=FAKE, qi=FAKE, R=2, tq=2, Hq=32, Hkv=8, D=128, P=16,
             scale=0.088, out=FAKE, lse=None, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    slh = (ctypes.c_int32 * 2)(*kw.get("seq", (17, 100)))
    qih = (ctypes.c_int32 * 3)(*kw.get("ind", (0, 1, 2)))
    return lib.pa_attention_varlen_q4(a["q"], a["k"], a["v"], a["nb"], a["bt"], a["mb"], a["sl"], a["qi"], slh, qih,
                                      a["R"], a["tq"], a["Hq"], a["Hkv"], a["D"], a["P"], a["scale"], a["out"],
                                      a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=64), b.PA_ERR_UNSUPPORTED),
    (dict(P=32), b.PA_ERR_UNSUPPORTED),
    (dict(Hq=16), b.PA_ERR_UNSUPPORTED),
    (dict(q=None), b.PA_ERR_INVALID_ARG),
    (dict(bt=None), b.PA_ERR_INVALID_ARG),
    (dict(out=ODD), b.PA_ERR_INVALID_ARG),
    (dict(k=ODD), b.PA_ERR_INVALID_ARG),
    (dict(ws=ctypes.c_void_p((1 << 20) + 16)), b.PA_ERR_INVALID_ARG),
    (dict(ind=(0, 1, 3)), b.PA_ERR_INVALID_ARG),
    (dict(ind=(0, 2, 1), tq=1), b.PA_ERR_INVALID_ARG),
    (dict(seq=(0, 100)), b.PA_ERR_INVALID_ARG),
    (dict(seq=(17, 1000)), b.PA_ERR_INVALID_ARG),
    (dict(ind=(0, 1, 9), tq=9, seq=(17, 7)), b.PA_ERR_INVALID_ARG),
    (dict(seq=(17, (1 << 20) + 1)), b.PA_ERR_UNSUPPORTED),
    (dict(wsb=1024, seq=(17, 600)), b.PA_ERR_WORKSPACE_TOO_SMALL),
    (dict(nb=0), b.PA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), b.PA_ERR_INVALID_ARG),
])
def test_attention_refusals(kw, status):
    n0 = lib.pa_launch_count()
    assert _attn(**kw) == status, lib.pa_last_error_message().decode()
    assert lib.pa_last_error_message().decode() != "" and lib.pa_launch_count() == n0


def test_the_binding_refuses_shapes_types_and_places():
    """Argument checks of the binding come before any call into the library;
    CPU tensors are themselves refused."""
    import torch
    pool = torch.zeros(4, 2, 1280, dtype=torch.uint8)
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    ws = torch.zeros(256, dtype=torch.uint8)
    for bad in [(rows, rows, slots[:2], pool, pool), (rows, rows[:2], slots, pool, pool),
                (rows, rows, slots, pool[..., :1152], pool[..., :1152]), (rows, rows, slots, pool, pool[:2])]:
        with pytest.raises(ValueError):
            b.pa_kv_append_q4(*bad, workspace=ws)
    with pytest.raises(ValueError):
        b.pa_kv_read_q4(slots[:, None], pool, pool, workspace=ws)
    with pytest.raises(ValueError):
        b.pa_kv_read_q4(slots, pool, pool, k_out=rows[:2], v_out=rows, workspace=ws)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    one = torch.ones(2, dtype=torch.int32)
    ind = torch.arange(3, dtype=torch.int32)
    tab = torch.zeros(2, 1, dtype=torch.int32)
    for kw in [dict(seq_lens_host=[1]), dict(qo_indptr_host=[0, 1]), dict(out=q[:1]),
               dict(lse=torch.zeros(2, 4))]:
        with pytest.raises(ValueError):
            b.pa_attention_varlen_q4(q, pool, pool, tab, one, ind, 0.1, workspace=ws, **kw)
    with pytest.raises(TypeError):
        b._data(rows, torch.uint8, "rows", 0)
    with pytest.raises(ValueError, match="current device"):
        b._data(rows, torch.bfloat16, "rows", 0)
    with pytest.raises(ValueError, match="contiguous"):
        b._data(rows.transpose(0, 1), torch.bfloat16, "rows", 0)
