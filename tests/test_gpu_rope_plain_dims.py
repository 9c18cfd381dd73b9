"""Dims behind rotary_dim are not rotated: without a norm they come out as they
went in, infinities, signed zeros and all, and an infinity there reaches nothing
else."""
import numpy as np
import pytest
import torch

from tests.test_gpu_norm_rope import DEV, Case
from tests.util import bf16_dev, bf16_host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from paged_kv_decode_varlen_gb300 import binding as B

VALUES = np.array([0x7f80, 0xff80, 0x8000, 0x0000, 0x7f7f, 0x0001, 0x8001], np.uint16)  # +-inf, +-0, the largest, tiny


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 32, 48, 64, 96, 112])
@pytest.mark.parametrize("append", [False, True])
def test_without_a_norm_they_stay(rotary, inter, append):
    c = Case(40, 3, rotary, inter, norm=False, seed=rotary)
    clean = [bf16_host(t) for t in c.plain()]
    rng = np.random.default_rng(1)
    for name in ("q", "k"):
        x = getattr(c, name).copy()
        at = rng.random(x.shape) < 0.2
        at[..., :rotary] = False
        x[at] = rng.choice(VALUES, x.shape)[at]
        setattr(c, name, x)
        setattr(c, "d" + name, bf16_dev(x))
    if append:
        kc = torch.zeros(3, 3, 16, 128, dtype=torch.bfloat16, device=DEV)
        vc, slots = torch.zeros_like(kc), np.arange(40)[::-1].copy()
        q = c.append(slots, kc, vc)
        got = [bf16_host(q), bf16_host(kc)[slots // 16, :, slots % 16]]
    else:
        got = [bf16_host(t) for t in c.plain()]
    for y, x, before in zip(got, (c.q, c.k), clean):
        assert np.array_equal(y[..., rotary:], x[..., rotary:])
        assert np.array_equal(y[..., :rotary], before[..., :rotary])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rotary", [0, 32, 112])
def test_with_a_norm_they_are_the_norm(rotary, inter):
    c = Case(20, 2, rotary, inter, seed=3)
    q, k = c.plain()
    none = B.pa_rope_turns([]).to(DEV)
    plain_q, plain_k = B.pa_qk_norm_rope(c.dq, c.dk, c.dpos, none, **c.kw_args)
    assert torch.equal(q[..., rotary:], plain_q[..., rotary:]) and torch.equal(k[..., rotary:], plain_k[..., rotary:])
