"""Inputs and error bounds of the 4-bit pool's tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import fp4

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def host(t: torch.Tensor) -> np.ndarray:
    """Any tensor's numbers on the host (floats as binary64)."""
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def rounded(x: np.ndarray, dtype: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype])


class Batch:
    """A filled 4-bit pool, scattered tables, ragged lengths and queries.  The
    pool starts as random bytes (NaN scales among them); only the sequences'
    own tokens are written, through the oracle."""

    def __init__(self, lens, heads, kv_heads, head, block, dtype="bf16", seed=0, key_scale=1.0,
                 value_scale=1.0, spare=3, query_std=1.0, width=None):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.dtype, self.scale = dtype, head ** -0.5
        self.key_scale, self.value_scale = key_scale, value_scale
        counts = -(-self.lens // block)
        blocks = int(counts.sum()) + spare
        perm = rng.permutation(blocks)
        width = max(1, int(counts.max(initial=0))) if width is None else width
        # unused table entries name no block: they must not be read
        self.tables = np.full((len(lens), width), 1 << 30, dtype=np.int32)
        at = 0
        for r, c in enumerate(counts):
            self.tables[r, :c] = perm[at:at + c]
            at += c
        self.cache = rng.integers(0, 256, (blocks, kv_heads, block // 8, 9 * head), dtype=np.uint8)
        self.slots = np.concatenate([self.tables[r, np.arange(n) // block].astype(np.int64) * block
                                     + np.arange(n) % block for r, n in enumerate(self.lens)] or
                                    [np.zeros(0, np.int64)]).astype(np.int64)
        n = len(self.slots)
        self.key = rounded(key_scale * rng.standard_normal((n, kv_heads, head)), dtype)
        self.value = rounded(value_scale * rng.standard_normal((n, kv_heads, head)), dtype)
        fp4.write(self.cache, host(self.key), host(self.value), self.slots, key_scale, value_scale)
        self.query = rounded(query_std * rng.standard_normal((len(lens), heads, head)), dtype)

    def reference(self):
        return fp4.decode(host(self.query), self.cache, self.tables, self.lens, self.scale,
                          self.key_scale, self.value_scale)


def decode_bound(ref, mass, total, reach, lens, head, dtype):
    """How far a decode's outputs may be off, by arithmetic.

    Scores: fp32 sums of head products in chains of head / 16 partial sums of
    16, each step off by at most 2^-22 of the sum's mass (a matrix unit may
    truncate), and one multiplication and subtraction: 2 * delta relative on a
    weight, delta = (head / 16 + 4) * 2^-22 * reach (plus the query's two
    fp16 parts for fp32 queries, 2^-22).  Weights: rounded to fp16, half a step
    2^-11 (bf16), or in two parts, 2^-22 (fp32); exp2 within 2^-22.  fp16 has no
    steps finer than 2^-24, so that a small weight is off by up to 2^-25 where
    the largest is kept at 2^7 or more: 2^-32 of the sum of |v|, which counts
    where the values of the large weights are zeros (4-bit values often are).
    Sums over tokens: a chain of length n / 16, each step 2^-23.  The result:
    half a step of its type, 2^-8 or 2^-24."""
    n = np.asarray(lens, dtype=np.float64).reshape(-1, 1, 1)
    delta = (head / 16 + 5) * 2.0 ** -22 * reach
    weight = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    out = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    return (2 * (2 * delta + weight + 2.0 ** -22 + (n / 16 + 16) * 2.0 ** -23) * mass
            + 2.0 ** -32 * total
            + out * (1 + 2.0 ** -6) * np.abs(ref) + 1e-30)


def assert_decode(got: torch.Tensor, batch: Batch, what=""):
    ref, mass, total, reach = batch.reference()
    g = host(got)
    assert np.isfinite(g).all(), what
    bound = decode_bound(ref, mass, total, reach, batch.lens, g.shape[-1], batch.dtype)
    worst = float(np.max(np.abs(g - ref) / bound, initial=0.0))
    assert worst <= 1.0, "%s: %.3g times the bound" % (what, worst)
    return worst
