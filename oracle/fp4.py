"""The 4-bit pool, its decode and the device-side tables in numpy and
binary64 -- TEST INFRASTRUCTURE ONLY, written from the definitions in
include/pa.h and sharing no code with the library.

A pool is uint8 [num_blocks, num_kv_heads, block_size / 8, 9 * D]; a tile (the
last axis) holds eight tokens: key codes [8][D / 2], value codes [D / 16][8][8],
key scales [8][D / 16], value scales [D / 16][8].
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
#: The non-negative e4m3 numbers in order: code c has exponent c >> 3 (bias 7)
#: and mantissa c & 7; exponent 0 is subnormal; code 127 is NaN.
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                 for c in range(127)])


def nearest_code(table: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the nearest entry of an ascending table, ties to the even
    index, past the end to the last."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    below, above = x - table[hi - 1], table[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(up, hi, hi - 1)


def quantise(x: np.ndarray, tensor_scale: float = 1.0):
    """Codes (0..15, bit 3 the sign) [..., D] and scale codes [..., D / 16] of
    numbers x [..., D] (any float type, taken as binary64)."""
    with np.errstate(invalid="ignore", over="ignore"):
        g = x.astype(np.float64).reshape(x.shape[:-1] + (-1, 16)) / tensor_scale
        top = np.abs(g).max(-1)
        nan = np.isnan(top)
        scale = nearest_code(E4M3, np.minimum(np.where(nan, 0.0, top) / 6.0, 448.0))
        s = E4M3[scale][..., None]
        q = np.where(s > 0, np.abs(g) / np.where(s > 0, s, 1.0), 0.0)
        code = nearest_code(E2M1, np.minimum(np.where(np.isnan(q), 0.0, q), 6.0))
        code = code + 8 * ((g < 0) & (code > 0))
    return code.reshape(x.shape).astype(np.uint8), np.where(nan, 0x7F, scale).astype(np.uint8)


def dequantise(codes: np.ndarray, scales: np.ndarray, tensor_scale: float = 1.0) -> np.ndarray:
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.append(E4M3, np.nan)[scales & 127] * tensor_scale
    return v * np.repeat(s, 16, axis=-1)


def _offsets(head_size: int, row: np.ndarray, values: bool):
    """Byte of every element's code [n, D] and of every group's scale [n, D / 16]
    in the tile, for rows [n]."""
    d, g, row = np.arange(head_size), np.arange(head_size // 16), np.asarray(row)[:, None]
    if values:
        return (4 * head_size + (d // 16) * 64 + row * 8 + (d % 16) // 2,
                8 * head_size + head_size // 2 + g * 8 + row)
    return row * (head_size // 2) + d // 2, 8 * head_size + row * (head_size // 16) + g


def read(cache: np.ndarray, slots, key_scale: float = 1.0, value_scale: float = 1.0):
    """Keys and values [n, num_kv_heads, D] of the slots."""
    _, hkv, tiles, size = cache.shape
    d = size // 9
    slots = np.asarray(slots, dtype=np.int64)
    block, off = slots // (8 * tiles), slots % (8 * tiles)
    rows = cache[block, :, off // 8]  # [n, hkv, 9 D]
    out = []
    for values, ts in ((False, key_scale), (True, value_scale)):
        code_at, scale_at = _offsets(d, off % 8, values)
        codes = np.take_along_axis(rows, np.repeat(code_at[:, None], hkv, 1), 2)
        codes = (codes >> (4 * (np.arange(d) % 2)).astype(np.uint8)) & 15
        scales = np.take_along_axis(rows, np.repeat(scale_at[:, None], hkv, 1), 2)
        out.append(dequantise(codes, scales, ts))
    return out


def write(cache: np.ndarray, key, value, slots, key_scale: float = 1.0, value_scale: float = 1.0):
    """Write tokens into the pool (in place); negative slots and slots past
    the pool are skipped."""
    nb, hkv, tiles, size = cache.shape
    d = size // 9
    for values, x, ts in ((False, key, key_scale), (True, value, value_scale)):
        codes, scales = quantise(x, ts)
        packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
        for t, slot in enumerate(np.asarray(slots)):
            if slot < 0 or slot >= nb * tiles * 8:
                continue
            tile = cache[slot // (8 * tiles), :, slot % (8 * tiles) // 8]
            code_at, scale_at = _offsets(d, [slot % 8], values)
            tile[:, code_at[0, 0::2]] = packed[t]
            tile[:, scale_at[0]] = scales[t]


def decode(query: np.ndarray, cache: np.ndarray, tables, lens, scale: float,
           key_scale: float = 1.0, value_scale: float = 1.0):
    """Decode attention [S, Hq, D] in binary64.  Also, per output element, the
    sum of weight * |value| and the sum of |value|, and, per row, the largest
    scale * sum |q_d k_d|, which bound rounding errors."""
    q = query.astype(np.float64)
    s, hq, d = q.shape
    hkv, bs = cache.shape[1], cache.shape[2] * 8
    group = hq // hkv
    out, mass, total = (np.zeros((s, hq, d)) for _ in range(3))
    reach = np.zeros((s, hq, 1))
    for r in range(s):
        n = int(lens[r])
        if n <= 0:
            continue
        pos = np.arange(n)
        slots = np.asarray(tables[r], dtype=np.int64)[pos // bs] * bs + pos % bs
        k, v = read(cache, slots, key_scale, value_scale)
        for h in range(hq):
            x = k[:, h // group] @ q[r, h] * scale
            w = np.exp(x - x.max())
            w /= w.sum()
            out[r, h] = w @ v[:, h // group]
            mass[r, h] = w @ np.abs(v[:, h // group])
            total[r, h] = np.abs(v[:, h // group]).sum(0)
            reach[r, h] = abs(scale) * (np.abs(k[:, h // group]) @ np.abs(q[r, h])).max()
    return out, mass, total, reach


def extend_tables(tables, lens, new, block_size, num_blocks, max_tokens, ring=None, state=None):
    """One step of the tables, request by request and token by token.
    Returns (tables, lens, state, slots, positions, starts, refused)."""
    tables, lens, new = np.array(tables), [int(x) for x in lens], [int(x) for x in new]
    state = None if state is None else [int(x) for x in state]
    before = (tables.copy(), list(lens), None if state is None else list(state))
    slots, positions, starts = [], [], [0]
    refused = any(n < 0 for n in new) or any(x < 0 for x in lens) or sum(new) > max_tokens
    for r, n in enumerate(new):
        if refused:
            break
        for _ in range(int(n)):
            p = lens[r]
            if p // block_size >= tables.shape[1]:
                refused = True
                break
            if p % block_size == 0 and ring is not None:
                if state[1] < 1:
                    refused = True
                    break
                tables[r, p // block_size] = ring[state[0]]
                state = [(state[0] + 1) % len(ring), state[1] - 1]
            b = int(tables[r, p // block_size])
            slots.append(b * block_size + p % block_size if 0 <= b < num_blocks else -1)
            positions.append(p)
            lens[r] = p + 1
        starts.append(len(slots))
    if refused:
        tables, lens, state = before
        slots, positions, starts = [], [], [0] * (len(new) + 1)
    pad = [-1] * (max_tokens - len(slots))
    return (tables, np.array(lens, dtype=np.int64), state, np.array(slots + pad, dtype=np.int64),
            np.array(positions + pad, dtype=np.int64), np.array(starts, dtype=np.int64), refused)
