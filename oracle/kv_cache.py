"""fp64 reference of the KV-cache operators (test infrastructure only; numpy, loops over blocks and rows).

Written from the definitions: the q4_0 format ("The economics of hybrid attention", table in "What a token of
context costs", gives its size), softmax weights per cached position, the choice of the positions that stay, and
the move of their rows.
"""
from __future__ import annotations

import numpy as np


def q4_0_quantise(x):
    """x [..., d] float (bf16 values): (codes [..., d] 0..15, scales [..., d/32] fp16)."""
    x = np.asarray(x, np.float64)
    xb = x.reshape(-1, 32)
    scales = np.zeros(xb.shape[0], np.float16)
    codes = np.full(xb.shape, 8, np.uint8)
    for i, row in enumerate(xb):
        if not np.all(np.isfinite(row)):
            scales[i] = np.nan
            continue
        m = row[np.argmax(np.abs(row))]  # argmax: the first of equals
        s = np.float16(np.clip(m / -8.0, -65504.0, 65504.0))
        if s == 0:
            continue
        scales[i] = s
        codes[i] = np.clip(np.rint(row / np.float64(s)) + 8, 0, 15)
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1] + (x.shape[-1] // 32,))


def q4_0_pack(codes):
    c = np.asarray(codes, np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def q4_0_values(packed, scales):
    """The numbers that a packed cache stands for, fp64."""
    p = np.asarray(packed, np.uint8)
    c = np.empty(p.shape[:-1] + (2 * p.shape[-1],), np.float64)
    c[..., 0::2] = (p & 15).astype(np.float64) - 8
    c[..., 1::2] = (p >> 4).astype(np.float64) - 8
    return c * np.repeat(np.asarray(scales, np.float16).astype(np.float64), 32, axis=-1)


def append(cache_values, cache_scales, x, cache_len, n_new):
    """Copies of one side's (packed, scales) cache with x [B,n,Hkv,d] appended."""
    vals, sc = cache_values.copy(), cache_scales.copy()
    T = vals.shape[1]
    for b in range(x.shape[0]):
        for i in range(min(max(int(n_new[b]), 0), x.shape[1])):
            pos = int(cache_len[b]) - min(max(int(n_new[b]), 0), x.shape[1]) + i
            if 0 <= pos < T:
                c, s = q4_0_quantise(x[b, i])
                vals[b, pos], sc[b, pos] = q4_0_pack(c), s
    return vals, sc


def decode(q, k, v, cache_len, gate, scale):
    """q, gate [B,Hq,d]; k, v [B,T,Hkv,d] fp64.  Returns (o [B,Hq,d], w [B,Hkv,T]: weights summed over the group)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    B, Hq, d = q.shape
    T, Hkv = k.shape[1], k.shape[2]
    g = Hq // Hkv
    o, w = np.zeros((B, Hq, d)), np.zeros((B, Hkv, T))
    for b in range(B):
        n = T if cache_len is None else min(max(int(cache_len[b]), 0), T)
        if n == 0:
            continue
        for h in range(Hq):
            s = scale * (k[b, :n, h // g] @ q[b, h])
            e = np.exp(s - s.max())
            p = e / e.sum()
            o[b, h] = p @ v[b, :n, h // g]
            w[b, h // g, :n] += p
    if gate is not None:
        o = o / (1 + np.exp(-np.asarray(gate, np.float64)))
    return o, w


def evict_select(acc, cache_len, n_keep, n_recent):
    acc = np.asarray(acc)
    B, H, T = acc.shape
    keep = np.full((B, H, n_keep), -1, np.int32)
    for b in range(B):
        n = T if cache_len is None else min(max(int(cache_len[b]), 0), T)
        for h in range(H):
            if n <= n_keep:
                keep[b, h, :n] = np.arange(n)
                continue
            old = n - n_recent
            # larger weight first (a NaN above all), then the lower position
            order = sorted(range(old), key=lambda j: (not np.isnan(acc[b, h, j]), -acc[b, h, j] if not
                                                      np.isnan(acc[b, h, j]) else 0.0, j))
            keep[b, h] = sorted(order[:n_keep - n_recent] + list(range(old, n)))
    return keep


def compact(array, keep, out):
    """array [B,T,H,...] -> a copy of out [B,Tout,H,...] with the kept rows in front."""
    res = out.copy()
    for b in range(keep.shape[0]):
        for h in range(keep.shape[1]):
            for i, j in enumerate(keep[b, h]):
                if 0 <= j < array.shape[1]:
                    res[b, i, h] = array[b, j, h]
    return res
