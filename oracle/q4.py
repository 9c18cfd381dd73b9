"""The q4 page format in plain numpy -- TEST INFRASTRUCTURE ONLY.

Quantises bf16 rows into slabs, and slabs back into the bf16 values their
codes stand for, one dim at a time by its place in the slab.  Attention over a
q4 pool is then the bf16 oracle on the unpacked pool, since the values are
bf16 numbers.
"""
from __future__ import annotations

import numpy as np

import oracle

DIM, PAGE, GROUP = 128, 16, 32
CODES = PAGE * DIM // 2
SLAB = CODES + PAGE * (DIM // GROUP) * 4


def round_bf16(x) -> np.ndarray:
    """fp64 -> bf16 bits, to nearest even, subnormal results kept (the page
    format's rounding; the attention oracle's flushes them)."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        _, e = np.frexp(x)
        ulp = np.ldexp(1.0, np.maximum(e - 8, -133))
        r = np.where(np.isfinite(x), np.rint(x / ulp) * ulp, x).astype(np.float32)
    r = np.where(np.abs(r) > np.float32(3.3895313892515355e+38), np.copysign(np.float32(np.inf), r), r)
    u = (np.ascontiguousarray(r, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7fc0), u)


def places(t: int):
    """(byte, shift) of every dim's code of token t in a slab."""
    d = np.arange(DIM)
    g, w, j = d // 32, d % 32 // 8, d % 8
    bit = 16 * (j % 2) + 4 * (j // 2)
    byte = 64 * t + 16 * (g ^ ((t >> 1) & 3)) + 4 * w + bit // 8
    return byte, (bit % 8).astype(np.uint8)


def quantize(bits: np.ndarray):
    """bf16 bits [..., 128] -> codes uint8 [..., 128], D bits and Z bits
    uint16 [..., 4]; binary32 operations in the documented order."""
    x = (bits.astype(np.uint32) << 16).view(np.float32).reshape(*bits.shape[:-1], DIM // GROUP, GROUP)
    lo, hi = x.min(-1), x.max(-1)
    f32 = np.float32
    d_bits = round_bf16(((hi - lo) / f32(15)) * f32(16))
    d = oracle.bf16_to_f64(d_bits).astype(f32)
    z_bits = round_bf16(lo - d)
    z = oracle.bf16_to_f64(z_bits).astype(f32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint(((x - z[..., None]) / d[..., None]) * f32(16) - f32(16))
    c = np.where(d[..., None] == 0, 0, np.clip(c, 0, 15))
    return c.reshape(bits.shape).astype(np.uint8), d_bits, z_bits


def append(new: np.ndarray, slots: np.ndarray, pool: np.ndarray):
    """Writes rows bf16 bits [N, H, 128] into a pool uint8 [nb, H, SLAB]."""
    codes, d, z = quantize(new)
    for i, slot in enumerate(slots):
        if slot < 0:
            continue
        blk, t = int(slot) // PAGE, int(slot) % PAGE
        byte, shift = places(t)
        for h in range(new.shape[1]):
            row = np.zeros(SLAB, np.uint8)
            np.bitwise_or.at(row, byte, codes[i, h] << shift)
            pool[blk, h, 64 * t:64 * t + 64] = row[64 * t:64 * t + 64]
            dz = np.stack([d[i, h], z[i, h]], -1).astype("<u2")
            pool[blk, h, CODES + 16 * t:CODES + 16 * t + 16] = dz.reshape(-1).view(np.uint8)


def unpack(pool: np.ndarray) -> np.ndarray:
    """Pool uint8 [nb, H, SLAB] -> the bf16 bits it stands for, [nb, H, 16, 128]."""
    nb, H, _ = pool.shape
    out = np.empty((nb, H, PAGE, DIM), np.float64)
    for t in range(PAGE):
        byte, shift = places(t)
        c = ((pool[..., byte] >> shift) & 15).astype(np.float64)
        dz = np.ascontiguousarray(pool[..., CODES + 16 * t:CODES + 16 * t + 16]).view("<u2").reshape(nb, H, 4, 2)
        d = np.repeat(oracle.bf16_to_f64(dz[..., 0]), GROUP, -1)
        z = np.repeat(oracle.bf16_to_f64(dz[..., 1]), GROUP, -1)
        with np.errstate(invalid="ignore", over="ignore"):
            out[:, :, t] = z + d * (1 + c / 16)
    return round_bf16(out)
