"""Inputs and error bounds of the 8-bit pool's tests."""
from __future__ import annotations

import numpy as np
import torch

from fp4_util import TORCH, host, rounded  # noqa: F401
from oracle import int8


class Batch:
    """A filled 8-bit pool, scattered tables, ragged lengths and queries.  The pool starts
    as random bytes (NaN scales among them); only the sequences' own blocks are written,
    through the oracle, from tokens whose size differs from block to block."""

    def __init__(self, lens, heads, kv_heads, head, block, dtype="bf16", seed=0, spare=3, query_std=1.0,
                 width=None, key=None, value=None, spread=0.5):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.dtype, self.scale, self.block = dtype, head ** -0.5, block
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
        self.cache = rng.integers(-128, 128, (blocks, kv_heads, block // 8, 16 * (head + 1)), dtype=np.int8)
        self.slots = np.concatenate([self.tables[r, np.arange(n) // block].astype(np.int64) * block
                                     + np.arange(n) % block for r, n in enumerate(self.lens)] or
                                    [np.zeros(0, np.int64)]).astype(np.int64)
        n = len(self.slots)
        size = np.exp(spread * rng.standard_normal((blocks, kv_heads)))[self.slots // block][..., None]
        self.key = rounded(rng.standard_normal((n, kv_heads, head)) if key is None else key, dtype)
        self.value = rounded(size * rng.standard_normal((n, kv_heads, head)) if value is None else value, dtype)
        int8.write(self.cache, host(self.key), host(self.value), self.slots)
        self.query = rounded(query_std * rng.standard_normal((len(lens), heads, head)), dtype)
        self.old = rng.random(self.tables.shape).astype(np.float32)

    def reference(self):
        return int8.decode(host(self.query), self.cache, self.tables, self.lens, self.scale)


def score_bound(reach, head):
    """Scores: fp32 sums of head products in chains of head / 16 partial sums of 16, each step
    off by at most 2^-22 of the sum's mass (a matrix unit may truncate), the products with
    the block's scale (two roundings), one subtraction; fp32 queries in two fp16 parts
    (2^-22)."""
    return (head / 16 + 7) * 2.0 ** -22 * reach


def decode_bound(ref, mass, total, reach, lens, head, dtype):
    """How far a decode's outputs may be off, by arithmetic.

    A weight is off by twice its score's error, 2^-22 of exp2, the product with the value
    scale (2^-24) and its rounding to fp16, half a step 2^-11 (bf16), or in two parts,
    2^-22 (fp32).  fp16 has no steps finer than 2^-24, so a small weight is off by up to
    2^-25 where the largest is kept at 2^7 or more, in units of the largest value scale
    rounded up to a power of two: 2^-31 of |code| times the largest scale.  Sums
    over tokens: a chain of length n / 16, each step 2^-23.  The result: half a step of its
    type, 2^-8 or 2^-24."""
    n = np.asarray(lens, dtype=np.float64).reshape(-1, 1, 1)
    weight = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    out = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    return (2 * (2 * score_bound(reach, head) + weight + 2.0 ** -21 + (n / 16 + 16) * 2.0 ** -23) * mass
            + 2.0 ** -31 * total
            + out * (1 + 2.0 ** -6) * np.abs(ref) + 1e-30)


def weights_bound(ref, old, reach, lens, head):
    """Sums of weights, which are not rounded to fp16: each twice its score's error for itself
    and for its row's sum, 2^-22 for either exp2, additions of n / 16 and of the heads and
    cells (at most 64) in a row; the old weights' product and sum."""
    n = np.asarray(lens, dtype=np.float64)[:, None]
    far = 2 * 2 * score_bound(reach, head)[:, :, 0].max(1, keepdims=True)
    return (far + (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -20) * ref + 2.0 ** -22 * np.abs(old) + 1e-30


def assert_decode(got: torch.Tensor, batch: Batch, what="", reference=None):
    ref, _, mass, total, reach = batch.reference() if reference is None else reference
    g = host(got)
    assert np.isfinite(g).all(), what
    bound = decode_bound(ref, mass, total, reach, batch.lens, g.shape[-1], batch.dtype)
    worst = float(np.max(np.abs(g - ref) / bound, initial=0.0))
    assert worst <= 1.0, "%s: %.3g times the bound" % (what, worst)
    return worst


def assert_weights(got: torch.Tensor, batch: Batch, before, decay, untouched, what="", reference=None):
    """got: the weights after a call, `before` those it added to, `untouched` what lay in the
    output behind the sequences' blocks."""
    _, ref, _, _, reach = batch.reference() if reference is None else reference
    g, old = host(got), decay * np.asarray(before, dtype=np.float64)
    mine = np.arange(g.shape[1]) < -(-np.maximum(batch.lens, 0)[:, None] // batch.block)
    bound = weights_bound(ref, old, reach, batch.lens, batch.query.shape[-1])
    assert np.array_equal(g[~mine], np.asarray(untouched, dtype=np.float64)[~mine]), what
    worst = float(np.max((np.abs(g - ref - old) / bound)[mine], initial=0.0))
    assert worst <= 1.0, "%s: weights %.3g times the bound" % (what, worst)
