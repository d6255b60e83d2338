"""Oracle of the paged prefix-KV cache -- TEST INFRASTRUCTURE ONLY.

A plain, slow, fp64 CPU statement of what include/mot_paged.h defines: the
power-of-two scaled e4m3 row, the norm + rotation + cache write of a ragged
chunk, and the attention of the chunk over its sequence's cached rows. Like
the other oracles it is imported only by ``tests/``; the library never imports
it and shares no code with it. The norm, rotation and attention are those of
the attention oracle (readings R2-R4) and of the prefix oracle (P2, P3).

Readings:
  C1 a cached row (one token, one head) in 8 bits is payload * 2^e with e the
     smallest integer, at least -64, such that amax <= 448 * 2^e, and the payload
     the e4m3 value nearest x * 2^-e (ties to the even mantissa); a row with an
     infinity or a NaN is NaN throughout.
  C2 query i of a chunk of n tokens in a sequence of L sits at position
     p = L - n + i and sees the keys j < max(visible, p + 1).
"""
from __future__ import annotations

import math

import numpy as np

from oracle.mot_attn_oracle import rms_norm_heads, rope_rotate

E4M3_MAX = 448.0


def round_to_e4m3(y: np.ndarray) -> np.ndarray:
    """|y| <= 448 to the nearest e4m3 value (bias 7, 3 mantissa bits, subnormals of 2^-9), ties to even."""
    y = np.asarray(y, dtype=np.float64)
    _, ex = np.frexp(np.abs(y))  # |y| = m 2^ex, m in [1/2, 1): binade 2^(ex - 1)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    return np.rint(y / step) * step


def quantise_rows(x: np.ndarray):
    """Rows [..., 128] -> (payload values, scales 2^e) per C1, NaN rows as NaN."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.max(np.abs(x), axis=-1)
    fine = np.isfinite(amax)
    e = np.full(amax.shape, -64, dtype=np.int64)
    for idx in np.ndindex(*amax.shape):
        if fine[idx]:
            while amax[idx] > math.ldexp(E4M3_MAX, int(e[idx])):
                e[idx] += 1
    scale = np.where(fine, np.ldexp(1.0, e), np.nan)
    with np.errstate(invalid="ignore"):
        payload = np.where(fine[..., None], round_to_e4m3(np.where(fine[..., None], x, 0.0) / np.ldexp(1.0, e)[..., None]),
                           np.nan)
    return payload, scale


def chunk_qkv(qkv: np.ndarray, positions, q_gain, k_gain, hq: int, hkv: int, eps: float, theta: float):
    """qkv [T, Hq + 2 Hkv, 128] -> (q^ [T, Hq, 128], k^ [T, Hkv, 128], v [T, Hkv, 128]), unrounded."""
    heads = np.moveaxis(np.asarray(qkv, dtype=np.float64), 1, 0)
    q = rope_rotate(rms_norm_heads(heads[:hq], q_gain, eps)[0], positions, theta)
    k = rope_rotate(rms_norm_heads(heads[hq:hq + hkv], k_gain, eps)[0], positions, theta)
    return np.moveaxis(q, 0, 1), np.moveaxis(k, 0, 1), np.moveaxis(heads[hq + hkv:], 0, 1)


def chunk_attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, visible: int):
    """q [n, Hq, 128] of the last n of L tokens, k, v [Hkv, L, 128].

    Returns (o [n, Hq, 128], lse [n, Hq], weighted |v| [n, Hq, 128], score
    magnitude [n, Hq]: the largest sum of |q_d k_d| / sqrt(128) over seen keys).
    Keys a query does not see have no influence whatever they hold.
    """
    n, hq, dh = q.shape
    hkv, length, _ = k.shape
    group = hq // hkv
    o = np.empty((n, hq, dh))
    lse = np.empty((n, hq))
    absv = np.empty((n, hq, dh))
    mag = np.empty((n, hq))
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(n):
            limit = max(int(visible), length - n + i + 1)
            for h in range(hq):
                kk, vv = k[h // group, :limit], v[h // group, :limit]
                s = (kk @ q[i, h]) / math.sqrt(dh)
                m = s.max()
                e = np.exp(s - m)
                den = e.sum()
                o[i, h] = (e / den) @ vv
                lse[i, h] = m + np.log(den)
                absv[i, h] = (e / den) @ np.abs(vv)
                mag[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() / math.sqrt(dh)
    return o, lse, absv, mag
