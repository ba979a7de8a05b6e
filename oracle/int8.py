"""The 8-bit pool, its decode, the eviction and the norms with rotation in numpy and
binary64 -- TEST INFRASTRUCTURE ONLY, written from the definitions in include/pa.h and
sharing no code with the library.

A pool is int8 [num_blocks, num_kv_heads, block_size / 8, 16 * (D + 1)]; a tile (the last
axis) holds eight tokens: two fp32 scales and 8 zeros, key codes plus 128 [D / 16][8][16],
value codes plus 128 likewise.
"""
from __future__ import annotations

import numpy as np


def scale_of(x: np.ndarray) -> np.ndarray:
    """max |x| / 127 as fp32 over the last two axes; NaN where x has no maximum."""
    with np.errstate(invalid="ignore"):
        top = np.abs(np.asarray(x, dtype=np.float64)).max((-2, -1))
        return np.where(np.isfinite(top), top / 127.0, np.nan).astype(np.float32)


def codes_of(x: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Nearest whole number of x / scale, ties to even; 0 where the scale is 0 or NaN."""
    s = np.broadcast_to(np.asarray(scale, dtype=np.float64), x.shape)
    ok = s > 0
    with np.errstate(invalid="ignore"):
        q = np.rint(np.where(ok, x, 0.0) / np.where(ok, s, 1.0))
    return np.clip(q, -127, 127).astype(np.int64)


def _tiles(cache: np.ndarray):
    _, _, tiles, size = cache.shape
    return tiles, size // 16 - 1


def block_codes(cache: np.ndarray, block: int, side: int) -> np.ndarray:
    """Codes [num_kv_heads, block_size, D] of a block (side 0: keys, 1: values)."""
    tiles, d = _tiles(cache)
    b = cache[block].view(np.uint8)[..., 16 + side * 8 * d:16 + (side + 1) * 8 * d]
    b = b.reshape(b.shape[0], tiles, d // 16, 8, 16).transpose(0, 1, 3, 2, 4)
    return b.reshape(b.shape[0], tiles * 8, d).astype(np.int64) - 128


def block_scales(cache: np.ndarray, block: int, side: int) -> np.ndarray:
    """Scales [num_kv_heads, tiles] of a block: equal over the tiles in a written one."""
    return np.ascontiguousarray(cache[block].view(np.uint8)[..., 4 * side:4 * side + 4]).view(np.float32)[..., 0]


def _put(cache, block, side, codes, scales):
    tiles, d = _tiles(cache)
    raw = cache.view(np.uint8)
    c = (codes + 128).astype(np.uint8).reshape(-1, tiles, 8, d // 16, 16).transpose(0, 1, 3, 2, 4)
    raw[block, :, :, 16 + side * 8 * d:16 + (side + 1) * 8 * d] = c.reshape(c.shape[0], tiles, 8 * d)
    s = np.ascontiguousarray(scales, dtype=np.float32).view(np.uint8).reshape(-1, 1, 4)
    raw[block, :, :, 4 * side:4 * side + 4] = s


def read(cache: np.ndarray, slots):
    """Keys and values [n, num_kv_heads, D] of the slots."""
    bs = cache.shape[2] * 8
    slots = np.asarray(slots, dtype=np.int64)
    out = [np.zeros((len(slots), cache.shape[1], _tiles(cache)[1])) for _ in range(2)]
    for block in np.unique(slots // bs):
        at = np.flatnonzero(slots // bs == block)
        for side in range(2):
            s = block_scales(cache, block, side)[:, slots[at] % bs // 8].astype(np.float64)
            c = block_codes(cache, block, side)[:, slots[at] % bs]
            out[side][at] = (c * s[..., None]).transpose(1, 0, 2)
    return out


def write(cache: np.ndarray, key, value, slots):
    """Write tokens into the pool (in place); negative slots and slots past the pool
    are skipped."""
    bs = cache.shape[2] * 8
    slots = np.asarray(slots, dtype=np.int64)
    live = np.flatnonzero((slots >= 0) & (slots < cache.shape[0] * bs))
    for block in np.unique(slots[live] // bs):
        at = live[slots[live] // bs == block]
        off = slots[at] % bs
        begins = bool((off == 0).any())
        for side, x in ((0, key), (1, value)):
            x = np.asarray(x)[at].astype(np.float64).transpose(1, 0, 2)  # [heads, tokens, D]
            codes, old = block_codes(cache, block, side), block_scales(cache, block, side)[:, 0]
            most = scale_of(x)
            scale = most if begins else np.where(np.isnan(old) | (most <= old), old, most)
            if not begins:
                grown = ~(most <= old) & ~np.isnan(old)
                again = codes_of(codes * old.astype(np.float64)[:, None, None], scale[:, None, None])
                codes = np.where(grown[:, None, None], again, codes)
            codes[:, off] = codes_of(x, scale[:, None, None])
            _put(cache, block, side, codes, scale)


def decode(query: np.ndarray, cache: np.ndarray, tables, lens, scale: float):
    """Decode attention [S, Hq, D] in binary64, and the attention of each block [S, width]
    summed over heads.  Also, per output element, the sum of weight * |value| and the sum of
    |code| times the sequence's largest value scale of the head, and, per row, the largest
    scale * sum |q_d k_d|, which bound rounding errors."""
    q = query.astype(np.float64)
    s, hq, d = q.shape
    hkv, bs = cache.shape[1], cache.shape[2] * 8
    group = hq // hkv
    out, mass, total = (np.zeros((s, hq, d)) for _ in range(3))
    reach = np.zeros((s, hq, 1))
    weights = np.zeros(np.asarray(tables).shape)
    for r in range(s):
        n = int(lens[r])
        if n <= 0:
            continue
        pos = np.arange(n)
        ids = np.asarray(tables[r], dtype=np.int64)[:-(-n // bs)]
        k, v = read(cache, ids[pos // bs] * bs + pos % bs)
        vs = np.stack([block_scales(cache, b, 1)[:, 0] for b in ids]).astype(np.float64)  # [blocks, heads]
        for h in range(hq):
            kv = h // group
            x = k[:, kv] @ q[r, h] * scale
            w = np.exp(x - x.max())
            w /= w.sum()
            out[r, h] = w @ v[:, kv]
            mass[r, h] = w @ np.abs(v[:, kv])
            some = np.where(vs[:, kv] > 0, vs[:, kv], 1.0)[pos // bs]
            total[r, h] = (np.abs(v[:, kv]) / some[:, None]).sum(0) * vs[:, kv].max()
            reach[r, h] = abs(scale) * (np.abs(k[:, kv]) @ np.abs(q[r, h])).max()
            weights[r, :len(ids)] += np.add.reduceat(w, np.arange(0, n, bs))
    return out, weights, mass, total, reach


def evict(tables, weights, lens, block_size, max_blocks, first, last, ring=None, state=None, gone=None):
    """One eviction, sequence by sequence.  Returns (tables, weights, lens, ring, state,
    gone, refused)."""
    tables, weights, lens = np.array(tables), np.array(weights), [int(x) for x in lens]
    ring = None if ring is None else np.array(ring)
    state = None if state is None else [int(x) for x in state]
    gone = None if gone is None else np.array(gone)
    before = (tables.copy(), weights.copy(), list(lens), None if ring is None else ring.copy(),
              None if state is None else list(state), None if gone is None else gone.copy())
    refused = any(n < 0 or -(-n // block_size) > tables.shape[1] for n in lens)
    if state is not None:
        refused |= not (0 <= state[0] < len(ring) and 0 <= state[1] <= len(ring))
    for r, length in enumerate(lens):
        n = -(-length // block_size)
        k = n - max_blocks
        if refused or k <= 0:
            continue
        w = [(np.isnan(weights[r, b]), 0.0 if np.isnan(weights[r, b]) else float(weights[r, b]) + 0.0, b)
             for b in range(first, n - last)]
        leave = sorted(b for _, _, b in sorted(w)[:k])
        left = set(leave)
        stay = [b for b in range(n) if b not in left]
        if state is not None:
            for b in leave:
                if state[1] == len(ring):
                    refused = True
                    break
                ring[(state[0] + state[1]) % len(ring)] = tables[r, b]
                state[1] += 1
        tables[r, :n] = tables[r, stay + leave]
        weights[r, :n] = np.concatenate([weights[r, stay], np.zeros(k, weights.dtype)])
        lens[r] -= k * block_size
        if gone is not None:
            gone[r] += k * block_size
    if refused:
        tables, weights, lens, ring, state, gone = before
    return tables, weights, np.array(lens, dtype=np.int64), ring, state, gone, refused


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """[n, heads, D] normed and rotated in binary64 (every position valid)."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if cos_sin is None:
        return y
    half = cos_sin.shape[1] // 2
    turn = np.asarray(cos_sin, dtype=np.float64)[np.asarray(positions)][:, None]
    out = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = turn[..., i], turn[..., half + i]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out
