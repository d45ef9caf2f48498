"""The 4-bit key-value cache in plain numpy, written from the header's
description of the format: levels, scales and lows on fp32 values, everything
that is summed in float64."""
import math

import numpy as np
import torch

GROUP = 32


def bf16_down(x):
    """fp32 values rounded down (towards -inf) to bf16, as fp32."""
    x = np.ascontiguousarray(x, np.float32)
    cut = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)       # towards zero
    more = ((x.view(np.uint32) & np.uint32(0xFFFF0000)).astype(np.uint64) + 0x10000)
    more = more.astype(np.uint32).view(np.float32)
    return np.where((cut > x), more, cut)


def quantise(x):
    """(levels [..., d] uint8, pairs [..., d / 32, 2] uint16: scale, low) of fp32 x [..., d]."""
    x = np.ascontiguousarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    levels = np.zeros(g.shape, np.uint8)
    pairs = np.zeros(g.shape[:-1] + (2,), np.uint16)
    with np.errstate(all="ignore"):
        low = bf16_down(g.min(-1)) + np.float32(0)
        span = g.max(-1) - low
        step = span * (np.float32(1) / np.float32(15))
        scale = -bf16_down(-step)
        bad = ~(np.isfinite(g).all(-1) & np.isfinite(span) & np.isfinite(scale))
        scale = np.where(span < np.float32(2.0 ** -100), np.float32(0), scale).astype(np.float32)
        inv = np.where(scale > 0, np.float32(1) / scale, np.float32(0)).astype(np.float32)
        lev = np.minimum(np.rint((g - low[..., None]) * inv[..., None]), 15)
    levels = np.where(bad[..., None], 0, lev).astype(np.uint8)
    pairs[..., 0] = np.where(bad, 0x7FC0, scale.view(np.uint32) >> 16)
    pairs[..., 1] = np.where(bad, 0x7FC0, low.astype(np.float32).view(np.uint32) >> 16)
    return levels.reshape(x.shape), pairs


def value_of(levels, pairs):
    """fp32 values [..., d]: low + scale * level, rounded once."""
    words = (pairs.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    lev = levels.reshape(*levels.shape[:-1], -1, GROUP).astype(np.float64)
    with np.errstate(all="ignore"):
        return (words[..., 1:2] + words[..., 0:1] * lev).reshape(levels.shape).astype(np.float32)


def place(c, off, d, values):
    """Byte and shift of channel c of the token `off` of a page, in its d / 2 bytes of levels."""
    g = c // GROUP
    if values:
        r, i = c % GROUP // 4, c % 4
        if d == 128 and (off >> 1) & 1:
            r ^= 4
        return r * (d // 16) + 2 * g + i // 2, 4 * (i % 2)
    q, i = c % GROUP // 8, c % 8
    return q * (d // 8) + 4 * g + i // 2, 4 * (i % 2)


def _maps(d, page, values):
    at = [[place(c, off, d, values) for c in range(d)] for off in range(page)]
    return np.array(at)[..., 0], np.array(at)[..., 1]                      # [page, d] each


def put_token(cache, page, head, side, off, x):
    """Write one token's row x [d] (fp32 values) into the numpy cache; returns what it stands for."""
    size, d = cache.shape[3], cache.shape[4] // 5 * 8
    rec = cache[page, head, side].reshape(-1)
    levels, pairs = quantise(x)
    row = np.zeros(d // 2, np.uint8)
    for c in range(d):
        byte, shift = place(c, off, d, side == 1)
        row[byte] |= levels[c] << shift
    rec[off * d // 2:(off + 1) * d // 2] = row
    at = size * d // 2 + off * d // 8
    rec[at:at + d // 8] = np.ascontiguousarray(pairs).view(np.uint8).reshape(-1)
    return value_of(levels, pairs)


def decode(cache):
    """fp32 [n_pages, Hkv, 2, page, d] of a numpy cache."""
    n, hkv, _, page, row = cache.shape
    d = row // 5 * 8
    flat = cache.reshape(n, hkv, 2, -1)
    out = np.empty((n, hkv, 2, page, d), np.float32)
    for side in (0, 1):
        packed = flat[:, :, side, :page * d // 2].reshape(n, hkv, page, d // 2)
        pairs = np.ascontiguousarray(flat[:, :, side, page * d // 2:]).view(np.uint16)
        byte, shift = _maps(d, page, side == 1)
        lev = (np.take_along_axis(packed, np.broadcast_to(byte, (n, hkv, page, d)), 3)
               >> shift.astype(np.uint8)) & 15
        out[:, :, side] = value_of(lev, pairs.reshape(n, hkv, page, d // GROUP, 2))
    return out


def tokens(decoded, table, n):
    """Keys and values [n, Hkv, d] of a sequence's first n tokens."""
    page = decoded.shape[3]
    rows = decoded[table[:-(-n // page)]] if n else decoded[:0]
    kv = rows.transpose(2, 0, 3, 1, 4).reshape(2, -1, decoded.shape[1], decoded.shape[4])[:, :n]
    return kv[0], kv[1]


def attend(decoded, q, table, lens, cu, scale=None, idx=None, cnt=None, block=0):
    """float64 o [Hq, T, d] and, for the tolerances, [Hq, T, 1] bounds: `size`, the largest |q| . |k| * scale
    over a row's tokens, and `span`, the largest |V| that it sees.  Rows of no sequence are 0."""
    hq, total, d = q.shape
    hkv = decoded.shape[1]
    scale = scale or 1 / math.sqrt(d)
    q = q.astype(np.float64)
    o, size, span = np.zeros((hq, total, d)), np.zeros((hq, total, 1)), np.zeros((hq, total, 1))
    for b, n in enumerate(lens):
        k, v = tokens(decoded, table[b], n)
        for h in range(hq):
            kh, vh = k[:, h // (hq // hkv)].astype(np.float64), v[:, h // (hq // hkv)].astype(np.float64)
            weight = np.ones(n)
            if idx is not None:
                hl = h // (hq // idx.shape[1])
                weight = np.zeros(n)
                for j in idx[b, hl, :cnt[b, hl]]:
                    if 0 <= j * block < n and j >= 0:
                        weight[j * block:(j + 1) * block] += 1
            for t in range(cu[b], cu[b + 1]):
                pos = n - cu[b + 1] + t
                sees = weight[:pos + 1] > 0 if pos >= 0 else np.zeros(0, bool)
                if not sees.any():
                    continue
                kk, vv, w = kh[:pos + 1][sees], vh[:pos + 1][sees], weight[:pos + 1][sees]
                s = kk @ q[h, t] * scale
                p = w * np.exp(s - s.max())
                o[h, t] = p @ vv / p.sum()
                size[h, t] = (np.abs(kk) @ np.abs(q[h, t]) * scale).max()
                span[h, t] = np.abs(vv).max()
    return o, size, span


def bf16(x):
    """numpy fp32 -> bf16 values, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().float().numpy()
