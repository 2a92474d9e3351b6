"""The 4-bit KV cache in plain numpy, 64 bits: quantisation by its definition, the
tile's layout by its formulas, attention, and derived error bounds (not collected as tests)."""

from __future__ import annotations

import math

import numpy as np
import torch

PAGE, TILE, GROUP = 64, 16, 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_toward(x, down):
    """The nearest fp16 not above (down) or not below x, as float64."""
    h = np.asarray(x, np.float64).astype(np.float16)
    over = h.astype(np.float64) > x if down else h.astype(np.float64) < x
    h = np.where(over, np.nextafter(h, np.float16(-np.inf if down else np.inf)), h)
    return h.astype(np.float64)


def quantise(x):
    """(codes, scales, minima) of rows [..., d] (float64)."""
    v = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    bad = ~(np.abs(v) <= 32768).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    z = half_toward(v.min(-1), True)
    s = half_toward((v.max(-1) - z) / 15, False)
    c = np.rint((v - z[..., None]) / np.where(s == 0, 1.0, s)[..., None])
    z, s = np.where(bad, np.nan, z), np.where(bad, np.nan, s)
    return c.reshape(x.shape), s, z


def values(c, s, z):
    return np.repeat(z, GROUP, -1) + np.repeat(s, GROUP, -1) * c


def quantised(x):
    return values(*quantise(x))


def offsets(d):
    """Byte of the code and of the scale and minimum of (row, value), K and V."""
    g_n = d // GROUP
    kb, ks, km, vb, vs, vm = (np.empty((TILE, d), np.int64) for _ in range(6))
    for r in range(TILE):
        for x in range(d):
            g, w, u = x // 32, x // 8, x // 4
            i = (r // 8) * g_n + w // 4
            kb[r, x] = 4 * ((i // 4) * 128 + ((r % 8) * 4 + w % 4) * 4 + i % 4) + (x % 8) // 2
            i = (u // 8) * 2 + r // 8
            vb[r, x] = 8 * d + 4 * ((i // 4) * 128 + ((u % 8) * 4 + (r % 8) // 2) * 4 + i % 4) + 2 * (r % 2) + (x % 4) // 2
            i = (r // 8) * g_n + g
            ks[r, x] = 16 * d + 4 * ((i // 4) * 16 + ((r % 8) // 2) * 4 + i % 4) + 2 * (r % 2)
            vs[r, x] = ks[r, x] + 2 * d
            km[r, x] = 17 * d + 2 * (r * g_n + g)
            vm[r, x] = 19 * d + 2 * (g * TILE + r)
    return kb, ks, km, vb, vs, vm


def unpack(pool, layer, pages, n):
    """K and V [n, kv heads, d] (float64) that the pool's bytes stand for; pool is numpy
    uint8 [layers, pages, kv heads, bytes], pages the sequence's page ids."""
    d = pool.shape[3] // (TILE * 5)
    raw = pool[layer, pages].reshape(len(pages), pool.shape[2], PAGE // TILE, 20 * d)
    raw = raw.transpose(0, 2, 1, 3).reshape(-1, pool.shape[2], 20 * d)  # [tile, head, bytes]
    kb, ks, km, vb, vs, vm = offsets(d)
    odd = np.arange(d) % 2 == 1
    half = np.ascontiguousarray(raw).view(np.float16)

    def get(b, s, m):
        code = np.where(odd, raw[:, :, b] >> 4, raw[:, :, b] & 15).astype(np.float64)
        out = half[:, :, m // 2].astype(np.float64) + half[:, :, s // 2].astype(np.float64) * code
        return out.transpose(0, 2, 1, 3).reshape(-1, pool.shape[2], d)[:n]

    return get(kb, ks, km), get(vb, vs, vm)


def tables(lens, rng, spare=2):
    """A block table with the pages in random order, and the number of pages of the pool."""
    n = [-(-v // PAGE) for v in lens]
    order = rng.permutation(sum(n) + spare).astype(np.int32)
    table = np.full((len(lens), max(max(n), 1)), 0, np.int32)
    at = 0
    for i, c in enumerate(n):
        table[i, :c] = order[at:at + c]
        at += c
    return table, sum(n) + spare


def attention(q, k, v, n_len, scale):
    """(out, reach) of the last rows q [n, heads, d] of a sequence with K, V [n_len, kv heads, d]
    (float64); reach[n, heads] = the largest scale * sum |q||k| of the positions seen."""
    n, heads, d = q.shape
    rep = heads // k.shape[1]
    out, reach = np.zeros((n, heads, d)), np.zeros((n, heads))
    for h in range(heads):
        kk, vv = k[:, h // rep], v[:, h // rep]
        for j in range(n):
            see = n_len - n + j + 1
            if see <= 0:
                continue
            s = kk[:see] @ q[j, h] * scale
            p = np.exp(s - s.max())
            out[j, h] = (p @ vv[:see]) / p.sum()
            reach[j, h] = np.abs(scale) * (np.abs(kk[:see]) @ np.abs(q[j, h])).max()
    return out, reach


def tolerance(out, reach, v_max, dtype):
    """Bound of |kernel - out| per element.

    A relative error e of every term of a score moves the score by at most
    e * reach, so every weight by a factor within exp(2 e reach) (numerator and sum).
    32-bit tensors: queries, weights and weight * scale as two fp16 parts (2^-21 or
    better together), fp32 sums: e = 2^-20 for the scores and for the weights.
    16-bit tensors: K and V rounded to fp16 for the matrix product of prompts
    (2^-11 each), queries exact in fp16 up to 2^-24 of the row's largest, weights fp16
    (2^-11), weight * scale once more (2^-11) where V is not rounded: scores 2^-11, weights
    and V or their scales together 2^-10.
    Then the output's own rounding, half a unit in the last place (2^-24 of v_max
    stands in for its subnormals in fp16)."""
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    e_s, e_p = (2.0**-20, 2.0**-20) if dtype == "fp32" else (2.0**-11, 2.0**-10)
    return eps * np.abs(out) + v_max * (np.expm1(2 * e_s * reach) + e_p)[..., None] + 2.0**-24


def default_scale(d):
    return 1.0 / math.sqrt(d)
