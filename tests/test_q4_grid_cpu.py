"""Where the q4 format's grid of a group ends, against the roundings of its D
and Z to bf16."""
import numpy as np
import pytest

import oracle
from oracle import q4
from paged_kv_decode_varlen_gb300 import workloads as W


@pytest.mark.parametrize("offset", [0.0, 1.0, 10.0, -300.0])
def test_the_ends_move_by_the_roundings_of_d_and_z(offset):
    rng = np.random.default_rng(17)
    x = rng.standard_normal((3000, 1, 128)) + offset
    bits = W.f32_to_bf16_bits(x.astype(np.float32))
    v = oracle.bf16_to_f64(bits).reshape(3000, 1, 4, 32)
    lo, hi = v.min(-1), v.max(-1)
    _, d, z = (oracle.bf16_to_f64(a) if a.dtype == np.uint16 else a for a in q4.quantize(bits))
    # 2^-8 each for Z and for D; binary32 rounds hi - lo, the quotient and lo - D, 2^-24 each
    z_off = (2.0 ** -8 + 2.0 ** -22) * np.abs(lo - d)
    assert np.all(np.abs(z + d - lo) <= z_off)
    assert np.all(np.abs(z + d * 31 / 16 - hi) <= z_off + (2.0 ** -8 + 2.0 ** -22) * (hi - lo))
    if offset == 0.0:
        # half of it (2^-9) is none: a number of significand m is off by up to 2^-8 / m of itself, and
        # those of lo - D take every value from 1 to 2 here (not at -300, where inputs lie 2 apart)
        assert np.any(np.abs(z + d - lo) > 0.5 * z_off)
