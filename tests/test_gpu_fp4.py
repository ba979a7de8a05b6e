"""The 4-bit pool on the GPU against the binary64 oracle: quantising write and
read-back (exact), block copies (exact), decode attention (within a bound
derived from the roundings), the device-side tables (exact), and the three as
a decode step, captured and replayed."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_78_gb300 as pa
from fp4_util import TORCH, Batch, assert_decode, decode_bound, host, rounded
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    pa.pa_get_device_error()
    yield


def dev(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).cuda()


def same(a, b):
    return np.array_equal(np.asarray(a, dtype=np.float64), b, equal_nan=True)


# ---------------------------------------------------------------------------
# write and read-back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,hkv,block,n", [(64, 1, 8, 1), (64, 3, 16, 77), (128, 8, 16, 130),
                                              (128, 2, 256, 300), (256, 5, 32, 41), (64, 1, 8, 1001),
                                              (64, 40, 16, 65), (128, 1, 16, 3), (256, 1, 8, 9)])
def test_write_and_gather(dtype, head, hkv, block, n):
    rng = np.random.default_rng(head + n)
    nb = -(-n // block) + 3
    cache = rng.integers(0, 256, (nb, hkv, block // 8, 9 * head), dtype=np.uint8)
    slots = rng.permutation(nb * block)[:n].astype(np.int64)
    k = rounded(4 * rng.standard_normal((n, hkv, head)) * np.exp(rng.standard_normal((n, hkv, 1))), dtype)
    v = rounded(0.1 * rng.standard_normal((n, hkv, head)), dtype)
    d = dev(cache)
    pa.pa_reshape_and_cache_fp4(d, dev(k), dev(v), dev(slots), 2.0, 0.125)
    want = cache.copy()
    fp4.write(want, host(k), host(v), slots, 2.0, 0.125)
    got = d.cpu().numpy()
    every = np.arange(nb * block)
    for a, b in zip(fp4.read(got, every, 2.0, 0.125), fp4.read(want, every, 2.0, 0.125)):
        assert same(a, b)
    # the read-back gives the very numbers, slots repeated
    again = np.concatenate([slots, slots[:3]])
    ko = torch.empty((len(again), hkv, head), dtype=TORCH[dtype], device="cuda")
    vo = torch.empty_like(ko)
    pa.pa_gather_cache_fp4(ko, vo, d, dev(again), 2.0, 0.125)
    rk, rv = fp4.read(want, again, 2.0, 0.125)
    assert same(host(ko), rk) and same(host(vo), rv)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_write_rounds_on_the_exact_quotients(dtype):
    # Every border of e2m1 times scales of every mantissa, the number itself
    # and its neighbours in the type; each group's maximum fixes its scale.
    rows = []
    for m in range(8, 16):
        for e in (-6, 0, 5):
            s = m / 8 * 2.0 ** e
            b = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * s
            t = torch.from_numpy(b.astype(np.float32)).to(TORCH[dtype])
            up = torch.nextafter(t, torch.full_like(t, float("inf")))
            down = torch.nextafter(t, torch.zeros_like(t))
            for x in (t, up, down):
                x = host(x)
                rows.append(np.concatenate([[6 * s], x, -x, [0.0]]))
    x = np.zeros((len(rows), 1, 64))
    x[:, 0, :16] = rows
    x[:, 0, 16:32] = np.array(rows)[:, ::-1]
    key, value = rounded(x, dtype), rounded(-x, dtype)
    cache = torch.zeros((-(-len(rows) // 8), 1, 1, 9 * 64), dtype=torch.uint8, device="cuda")
    slots = torch.arange(len(rows), device="cuda")
    pa.pa_reshape_and_cache_fp4(cache, dev(key), dev(value), slots)
    gk, gv = fp4.read(cache.cpu().numpy(), np.arange(len(rows)))
    assert same(gk, fp4.dequantise(*fp4.quantise(host(key))))
    assert same(gv, fp4.dequantise(*fp4.quantise(host(value))))


def test_write_rounds_fp32_numbers_near_borders():
    """Numbers beside the borders of e2m1, nearer and nearer, in groups without any
    whose quotient is a multiple of 1/4; then with one such in every other group."""
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for k in range(9, 24):
        for m in range(8, 16):
            s, d = m / 8 * 2.0 ** (m % 3 - 1), 2.0 ** -k
            rows.append(np.concatenate([[6.01 * s], border * (1 + d) * s, -border * (1 - d) * s, [0.3 * s]]))
            rows.append(np.concatenate([[6.01 * s], border * (1 - d) * s, -border * (1 + d) * s, [0.5 * s]]))
    x = rounded(np.array(rows).reshape(-1, 1, 64), "fp32")
    n = x.shape[0]
    cache = torch.zeros((-(-n // 8), 1, 1, 9 * 64), dtype=torch.uint8, device="cuda")
    pa.pa_reshape_and_cache_fp4(cache, dev(x), dev(-x), torch.arange(n, device="cuda"))
    gk, gv = fp4.read(cache.cpu().numpy(), np.arange(n))
    want = fp4.dequantise(*fp4.quantise(host(x)))
    assert same(gk, want) and same(gv, -want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_write_special_values(dtype):
    rng = np.random.default_rng(7)
    x = rng.standard_normal((6, 2, 64))
    x[0, 0, 3] = np.nan
    x[1, 1, 17] = np.inf
    x[2, 0, 40] = -np.inf
    x[2, 0, 41] = np.nan
    x[3] = 0.0
    x[4] = 1e-30 * rng.standard_normal((2, 64))     # below the smallest scale
    x[5] = 3e38 * np.sign(rng.standard_normal((2, 64)))
    t = rounded(x, dtype)
    cache = torch.randint(0, 256, (1, 2, 1, 9 * 64), dtype=torch.uint8, device="cuda")
    pa.pa_reshape_and_cache_fp4(cache, dev(t), dev(t), torch.arange(6, device="cuda"))
    want = fp4.dequantise(*fp4.quantise(host(t)))
    for got in fp4.read(cache.cpu().numpy(), np.arange(6)):
        assert same(got, want)
    ko = torch.empty((6, 2, 64), dtype=TORCH[dtype], device="cuda")
    vo = torch.empty_like(ko)
    pa.pa_gather_cache_fp4(ko, vo, cache, torch.arange(6, device="cuda"))
    assert same(host(ko), want) and same(host(vo), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tensor_scale", [0.5, 0.25, 1.0, 2.0 ** -32, 2.0 ** 32])
def test_write_saturates_under_every_tensor_scale(dtype, tensor_scale):
    """Infinities, and finite numbers below and above what the largest scale holds and
    what 32 bits hold once divided by the tensor scale."""
    rng = np.random.default_rng(17)
    big = np.array([2688.0, 2689.0, 2700.0, 3e4, 1e20, 1e38, 3.3e38, 3.5e38, 1e40, 1e47]) * tensor_scale
    big = np.append(big[big < 3.38e38], [2.0 ** 127, 3.38e38, np.inf, np.nan])
    x = rng.standard_normal((len(big), 2, 64)) * tensor_scale
    x[:, 0, 5], x[:, 1, 20] = big, -big
    x[-1, 0, 6] = np.inf                  # beside a NaN
    t = rounded(x, dtype)
    n = len(big)
    cache = torch.randint(0, 256, (-(-n // 8), 2, 1, 9 * 64), dtype=torch.uint8, device="cuda")
    slots = torch.arange(n, device="cuda")
    pa.pa_reshape_and_cache_fp4(cache, dev(t), dev(-t), slots, tensor_scale, tensor_scale)
    want = fp4.dequantise(*fp4.quantise(host(t), tensor_scale), tensor_scale)
    k, v = fp4.read(cache.cpu().numpy(), np.arange(n), tensor_scale, tensor_scale)
    assert same(k, want) and same(v, -want)
    assert np.isnan(want[-1, 0, :16]).all() and np.isfinite(want[:-1]).all()


def test_padding_and_slots_outside_the_pool():
    rng = np.random.default_rng(8)
    cache = rng.integers(0, 256, (3, 2, 2, 9 * 64), dtype=np.uint8)
    k = rounded(rng.standard_normal((5, 2, 64)), "bf16")
    slots = np.array([5, -1, 48, 47, 1 << 40], dtype=np.int64)
    d = dev(cache)
    pa.pa_reshape_and_cache_fp4(d, dev(k), dev(k), dev(slots))
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SLOT
    want = cache.copy()
    fp4.write(want, host(k), host(k), slots)
    others = np.setdiff1d(np.arange(48), [5, 47])
    for a, b in zip(fp4.read(d.cpu().numpy(), others), fp4.read(cache, others)):
        assert same(a, b)
    ko = torch.full((5, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 8.0)
    pa.pa_gather_cache_fp4(ko, vo, d, dev(slots))
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SLOT
    rk, rv = fp4.read(want, slots[[0, 3]])
    assert same(host(ko)[[0, 3]], rk) and same(host(vo)[[0, 3]], rv)
    assert (host(ko)[[1, 2, 4]] == 9).all() and (host(vo)[[1, 2, 4]] == 8).all()


def test_write_takes_rows_of_a_fused_projection():
    rng = np.random.default_rng(9)
    qkv = dev(rounded(rng.standard_normal((37, 6 * 64)), "bf16"))
    k, v = qkv[:, 2 * 64:4 * 64].unflatten(1, (2, 64)), qkv[:, 4 * 64:].unflatten(1, (2, 64))
    slots = torch.arange(37, device="cuda")
    a, b = (pa.alloc_fp4_cache(5, 8, 2, 64) for _ in range(2))
    pa.pa_reshape_and_cache_fp4(a, k, v, slots)
    pa.pa_reshape_and_cache_fp4(b, k.contiguous(), v.contiguous(), slots)
    assert torch.equal(a, b) and a.any()
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache_fp4(a, k.transpose(1, 2).contiguous().transpose(1, 2), v, slots)
    with pytest.raises(pa.PAError):  # rows that start off a 16-byte boundary
        pa.pa_reshape_and_cache_fp4(a, qkv[:, 1:129].unflatten(1, (2, 64)), v, slots)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,hkv", [(64, 3), (128, 2), (256, 1)])
def test_write_and_gather_rows_off_32_byte_boundaries(dtype, head, hkv):
    """Rows that start 16 bytes into an allocation, and strides and outputs likewise."""
    rng = np.random.default_rng(head)
    n, half = 37, 8 if dtype == "bf16" else 4                  # elements of 16 bytes
    slots = rng.permutation(48)[:n].astype(np.int64)
    for off, odd in ((half, 0), (0, half), (half, half)):
        stride = hkv * head + odd
        kv = [dev(rounded(rng.standard_normal(n * stride + half), dtype)) for _ in range(2)]
        key, value = (x.as_strided((n, hkv, head), (stride, head, 1), off) for x in kv)
        cache = torch.zeros((3, hkv, 2, 9 * head), dtype=torch.uint8, device="cuda")
        pa.pa_reshape_and_cache_fp4(cache, key, value, dev(slots), 0.5, 2.0)
        k, v = fp4.read(cache.cpu().numpy(), slots, 0.5, 2.0)
        assert same(k, fp4.dequantise(*fp4.quantise(host(key), 0.5), 0.5))
        assert same(v, fp4.dequantise(*fp4.quantise(host(value), 2.0), 2.0))
        size = n * hkv * head
        for at, bt in ((half, half), (0, half), (half, 0)):    # one of the outputs, or both
            flat = torch.full((2, size + 2 * half), 7.0, dtype=TORCH[dtype], device="cuda")
            ko, vo = flat[0, at:at + size], flat[1, bt:bt + size]
            pa.pa_gather_cache_fp4(ko.view(n, hkv, head), vo.view(n, hkv, head), cache, dev(slots), 0.5, 2.0)
            assert same(host(ko).reshape(k.shape), k) and same(host(vo).reshape(v.shape), v)
            for row, x in ((flat[0], at), (flat[1], bt)):
                assert (row[:x] == 7).all() and (row[x + size:] == 7).all()


def test_no_tokens():
    c = pa.alloc_fp4_cache(2, 8, 2, 64)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    pa.pa_reshape_and_cache_fp4(c, k, k, s)
    pa.pa_gather_cache_fp4(k, k, c, s)


@pytest.mark.parametrize("head,hkv,block", [(64, 1, 8), (128, 3, 16), (256, 2, 64)])
def test_block_copies(head, hkv, block):
    rng = np.random.default_rng(head)
    a = rng.integers(0, 256, (9, hkv, block // 8, 9 * head), dtype=np.uint8)
    d = dev(a)
    pairs = torch.tensor([[0, 7], [3, 1], [8, 2]], device="cuda")
    pa.pa_copy_blocks(d, pairs)
    want = a.copy()
    want[[7, 1, 2]] = a[[0, 3, 8]]
    assert np.array_equal(d.cpu().numpy(), want)
    cpu = torch.zeros((4, hkv, block // 8, 9 * head), dtype=torch.uint8).pin_memory()
    pa.pa_swap_blocks(cpu, d, torch.tensor([[7, 3], [4, 0]], device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(cpu.numpy()[[3, 0]], want[[7, 4]]) and not cpu[1:3].any()
    pa.pa_swap_blocks(d, cpu, torch.tensor([[3, 5]], device="cuda"))
    want[5] = want[7]
    assert np.array_equal(d.cpu().numpy(), want)
    pa.pa_copy_blocks(d, torch.tensor([[0, 9]], device="cuda"))
    assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(d.cpu().numpy(), want)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

class Run:
    """A batch on the device and its decode."""

    def __init__(self, batch, workspace=None):
        b = self.batch = batch
        self.cache, self.query = dev(b.cache), dev(b.query)
        self.tables, self.lens = dev(b.tables), dev(b.lens)
        self.out = torch.full_like(self.query, 77.0)
        self.ws = workspace
        if workspace is None:
            self.ws = pa.alloc_workspace(pa.pa_decode_fp4_workspace_size(self.cache, b.query.shape[1]),
                                         "cuda")

    def __call__(self, stream=None):
        b = self.batch
        pa.pa_decode_fp4(self.out, self.query, self.cache, self.tables, self.lens, b.scale, self.ws,
                         b.key_scale, b.value_scale, stream=stream)
        return self.out


EDGES = [0, 1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 0, 255, 257, 500]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,block", [(64, 8), (64, 16), (128, 8), (128, 16), (128, 64), (256, 16),
                                        (256, 256), (64, 128)])
def test_decode_edge_lengths(dtype, head, block):
    r = Run(Batch(EDGES, 8, 2, head, block, dtype, seed=head + block))
    assert_decode(r(), r.batch)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("group", list(range(1, 17)))
@pytest.mark.parametrize("head", [64, 128, 256])
def test_decode_groups(head, group):
    hkv = 1 + group % 3
    for dtype in ("bf16", "fp32"):
        r = Run(Batch([3, 100, 45], hkv * group, hkv, head, 16, dtype, seed=group))
        assert_decode(r(), r.batch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,heads,hkv,head,block", [
    ([4096], 8, 1, 128, 16),              # one pair over many CTAs
    ([5000, 1, 0, 3001], 4, 4, 64, 16),
    ([20001], 16, 1, 64, 32),
    ([2500, 777], 12, 2, 256, 8),
    ([300] * 40, 40, 40, 128, 16),        # more pairs than CTAs
    (list(range(0, 900, 7)), 7, 1, 128, 8),
])
def test_decode_larger(lens, heads, hkv, head, block, dtype):
    r = Run(Batch(lens, heads, hkv, head, block, dtype, seed=len(lens)))
    first = r().clone()
    assert_decode(first, r.batch)
    # again on the same workspace, and the same bits
    r.out.fill_(55.0)
    assert torch.equal(r(), first)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_peaked_and_scaled(dtype):
    # large scores (weights close to 0 and 1), tensor scales, large queries
    r = Run(Batch([50, 700, 33], 6, 2, 128, 16, dtype, seed=5, key_scale=4.0, value_scale=2.0 ** -6,
                  query_std=30.0))
    assert_decode(r(), r.batch)
    r = Run(Batch([50, 700, 33], 6, 2, 128, 16, dtype, seed=6, query_std=2.0 ** -40))
    assert_decode(r(), r.batch)
    r = Run(Batch([50, 700, 33], 6, 2, 128, 16, dtype, seed=7, key_scale=2.0 ** -30, query_std=2.0 ** 30))
    assert_decode(r(), r.batch)
    b = Batch([64, 90], 4, 2, 64, 16, dtype, seed=8)
    b.scale = -0.3
    assert_decode(Run(b)(), b)
    b.scale = 0.0
    assert_decode(Run(b)(), b)


def test_decode_rising_scores():
    # the running maximum moves at every tile, by more and more
    b = Batch([600], 4, 1, 64, 16, "bf16", seed=9)
    ramp = np.linspace(0.0, 60.0, 600)[:, None, None] * np.ones((1, 1, 64))
    fp4.write(b.cache, ramp, host(b.value), b.slots)
    b.query = torch.ones_like(b.query)
    assert_decode(Run(b)(), b)
    fp4.write(b.cache, ramp[::-1], host(b.value), b.slots)
    assert_decode(Run(b)(), b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("far,tokens,seqs", [(40, 100, 1), (3000, 5000, 1), (4999, 5000, 1), (70, 90, 400)])
def test_decode_scores_below_the_least_number_weigh_nothing(dtype, far, tokens, seqs):
    """The first `far` tokens' scores are beyond 32 bits, the others' are zero: the mean of
    the others' values, whose weights are equal and exact.  Off are sums (2^-23 an addition
    of 16 tokens) and the output's rounding."""
    b = Batch([tokens], 4, 2, 64, 16, dtype, seed=far)
    key = np.zeros((tokens, 2, 64))
    key[:far] = 6 * 448.0
    fp4.write(b.cache, key, host(b.value), b.slots)
    b.query = rounded(np.full((1, 4, 64), -(2.0 ** 120)), dtype)
    ref, mass = b.reference()[:2]
    r = Run(b)
    r.tables, r.lens = r.tables.expand(seqs, -1).contiguous(), r.lens.expand(seqs).contiguous()
    r.query = r.query.expand(seqs, -1, -1).contiguous()
    r.out = torch.full_like(r.query, 77.0)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    bound = half * (1 + 2.0 ** -6) * np.abs(ref) + (tokens / 16 + 16) * 2.0 ** -23 * mass
    assert (np.abs(host(r()) - ref) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 20, 2.0 ** 24, 2.0 ** 27, 2.0 ** 34, 2.0 ** 60, 2.0 ** 110])
def test_decode_scores_with_steps_above_one(dtype, size):
    """Scores so large that neighbouring fp32 numbers are units or more apart: the token with
    the largest has all the weight (the next is further away than scores are off: a sum
    of head / 16 + 5 parts, 2^-22 of its mass each, twice), which is rounded once to fp16."""
    b = Batch([700, 33, 5000], 6, 2, 64, 16, dtype, seed=31, query_std=size)
    ref, _, _, reach = b.reference()
    sure = np.zeros(ref.shape[:2], dtype=bool)
    for r, n in enumerate(b.lens):
        at = np.arange(n)
        k, v = fp4.read(b.cache, b.tables[r, at // 16].astype(np.int64) * 16 + at % 16)
        for h in range(6):
            x = np.sort(k[:, h // 3] @ host(b.query)[r, h]) * b.scale
            sure[r, h] = x[-1] - x[-2] > 2 * 9 * 2.0 ** -22 * reach[r, h, 0] + 40
    assert sure.sum() >= 12
    got = host(Run(b)())
    half = 2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    assert np.isfinite(got).all()
    assert (np.abs(got - ref)[sure] <= half * np.abs(ref)[sure] + 1e-12).all()


def test_decode_nan_and_infinity():
    b = Batch([40, 60, 50], 4, 2, 64, 16, "bf16", seed=10)
    q = b.query.clone()
    q[0, 1, 5] = float("nan")
    q[2, 3, 9] = float("inf")
    b.query = q
    # a NaN key of sequence 1's first KV head, token 20
    slot = b.slots[40 + 20]
    k, v = fp4.read(b.cache, [slot])
    k[0, 0, 3] = np.nan
    fp4.write(b.cache, k, v, [slot])
    r = Run(b)
    got = host(r())
    bad = np.zeros(got.shape, dtype=bool)
    bad[0, 1] = bad[2, 3] = bad[1, :2] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_decode_takes_strided_queries_and_padded_tables():
    b = Batch([5, 60, 33], 6, 2, 128, 16, seed=11, width=40)
    r = Run(b)
    wide = torch.randn((3, 10 * 128), device="cuda").bfloat16()
    wide[:, 128:7 * 128] = r.query.flatten(1)
    r.query = wide[:, 128:7 * 128].unflatten(1, (6, 128))
    assert not r.query.is_contiguous()
    assert_decode(r(), b)
    with pytest.raises(ValueError):
        pa.pa_decode_fp4(r.out, r.query.transpose(0, 1).contiguous().transpose(0, 1), r.cache,
                         r.tables, r.lens, b.scale, r.ws)
    with pytest.raises(ValueError):
        pa.pa_decode_fp4(r.out[:, :, ::2], r.query[:, :, ::2], r.cache, r.tables, r.lens, b.scale, r.ws)


def test_decode_length_errors_touch_nothing_else():
    b = Batch([16, 40, 8], 4, 2, 64, 16, seed=12, width=3)
    r = Run(b)
    r.lens[0] = 49                       # three blocks hold 48
    got = r()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    ref = b.reference()[0]
    assert np.abs(host(got)[1:] - ref[1:]).max() < 0.05
    r.lens[0] = -4                       # as an empty sequence
    r.lens[1] = (1 << 31) - 1
    got = r()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    assert not got[0].any() and np.abs(host(got)[2] - ref[2]).max() < 0.05


def test_decode_block_ids_outside_the_pool_count_as_zeros():
    b = Batch([48, 20], 4, 2, 64, 16, seed=13)
    r = Run(b)
    for bad in (-1, b.cache.shape[0], -(1 << 31), (1 << 31) - 1):
        r.tables[0, 1] = bad
        got = host(r())
        assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID
        z = Batch([48, 20], 4, 2, 64, 16, seed=13)
        fp4.write(z.cache, np.zeros((16, 2, 64)), np.zeros((16, 2, 64)),
                  z.tables[0, 1].astype(np.int64) * 16 + np.arange(16))
        assert_decode(r.out, z)
        assert np.isfinite(got).all()


@pytest.mark.parametrize("head,heads", [(64, 4), (128, 8)])
def test_decode_bad_ids_among_the_last_stages(head, heads):
    """Zeros that lanes write themselves, in stages that no later copy follows."""
    tokens, shape = 500, dict(heads=heads, kv_heads=1, head=head, block=8, seed=32)
    r = Run(Batch([tokens], **shape))
    for bad in [(60,), (61, 62), (50, 56), tuple(range(40, 63)), tuple(range(0, 63, 3))]:
        z = Batch([tokens], **shape)
        for i in bad:
            fp4.write(z.cache, np.zeros((8, 1, head)), np.zeros((8, 1, head)),
                      z.tables[0, i].astype(np.int64) * 8 + np.arange(8))
        r.tables = dev(z.tables)
        r.tables[0, list(bad)] = -1
        for _ in range(3):
            assert_decode(r(), z, bad)
        assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID


def test_decode_rows_behind_the_batch_stay():
    b = Batch([30, 0, 70], 4, 2, 64, 16, seed=14)
    r = Run(b)
    big = torch.full((5, 4, 64), 33.0, dtype=torch.bfloat16, device="cuda")
    r.out = big[:3]
    before = r.cache.clone()
    assert_decode(r(), b)
    assert (big[3:] == 33).all() and torch.equal(before, r.cache)


def test_decode_past_32_bit_offsets():
    # a pool of more than 4 GB; the sequence's blocks lie at its end
    blocks = 260_000
    cache = torch.zeros((blocks, 8, 2, 9 * 128), dtype=torch.uint8, device="cuda")
    b = Batch([100], 16, 8, 128, 16, seed=15, spare=0)
    first = blocks - b.cache.shape[0]
    cache[first:] = dev(b.cache)
    r = Run(b)
    r.cache = cache
    r.tables = dev(np.where(b.tables < (1 << 30), b.tables + first, b.tables).astype(np.int32))
    assert_decode(r(), b)
    ko = torch.empty((100, 8, 128), dtype=torch.float32, device="cuda")
    vo = torch.empty_like(ko)
    slots = dev(b.slots + first * 16)
    pa.pa_gather_cache_fp4(ko, vo, cache, slots)
    rk, rv = fp4.read(b.cache, b.slots)
    assert same(host(ko), rk) and same(host(vo), rv)
    pa.pa_reshape_and_cache_fp4(cache, vo, ko, slots)
    pa.pa_gather_cache_fp4(ko, vo, cache, slots)
    assert same(host(ko), fp4.dequantise(*fp4.quantise(rv)))
    assert not cache[:first].any()


def test_decode_many_sequences():
    lens = [1 + (i * 7) % 19 for i in range(3001)]
    r = Run(Batch(lens, 2, 1, 64, 8, seed=16))
    assert_decode(r(), r.batch)


def test_decode_most_sequences():
    lens = [(i // 17) % 11 if i % 17 == 0 or i == 65534 else 0 for i in range(65535)]
    r = Run(Batch(lens, 2, 2, 64, 8, seed=24))
    assert_decode(r(), r.batch)


@pytest.mark.parametrize("head,heads,hkv", [(64, 4, 2), (128, 2, 2), (256, 3, 3)])
@pytest.mark.parametrize("most,long", [(40, 0), (200, 0), (40, 9000), (300, 5000)])
def test_decode_short_sequences_beside_long_ones(head, heads, hkv, most, long):
    """Pairs that stay whole with a warp or a CTA, next to ones that are cut."""
    rng = np.random.default_rng(most + long + head)
    lens = rng.integers(0, most, 1500 if most < 100 else 300)
    lens[7::31] = 0
    if long:
        lens[[0, 150, len(lens) - 1]] = long, long - 3, long // 2
    r = Run(Batch(lens, heads, hkv, head, 16, seed=head + most))
    assert_decode(r(), r.batch)


@pytest.mark.parametrize("head,heads,hkv", [(64, 8, 8), (128, 4, 4), (256, 5, 5)])
@pytest.mark.parametrize("longest", [510, 530, 1100])
def test_decode_pairs_about_as_long_as_may_stay_whole(head, heads, hkv, longest):
    rng = np.random.default_rng(longest + head)
    lens = rng.choice([1, 60, 480, 511, 512, 513, longest], 700, p=[.3, .3, .08, .08, .08, .08, .08])
    b = Batch([max(lens)], heads, hkv, head, 16, seed=head + longest)
    b.tables, b.lens = b.tables.repeat(len(lens), 0), lens.astype(np.int32)
    b.query = rounded(rng.standard_normal((len(lens), heads, head)), "bf16")
    assert_decode(Run(b)(), b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_sequences_that_share_blocks_and_repeated_calls(dtype):
    """Rows of one table several times over, and calls that agree bit for bit
    however the parts of a sequence arrive."""
    b = Batch([5000, 77], 12, 2, 128, 16, dtype, seed=25)
    b.tables, b.lens = b.tables[[0, 1, 0, 0, 1]], b.lens[[0, 1, 0, 0, 1]]
    b.lens[3] = 4000
    b.query = rounded(np.random.default_rng(26).standard_normal((5, 12, 128)), dtype)
    r = Run(b)
    first = r().clone()
    assert_decode(first, b)
    for _ in range(20):
        assert torch.equal(r(), first)


def test_decode_fp32_sums_are_rounded_not_cut_off():
    """512 sequences of 30000 tokens, so that a warp's share of one is over 10000
    tokens, and values of one sign.  Additions to a running sum that round to
    nearest are off by 2^-24 / sqrt(3) of it at most, in standard deviation, and
    either way: n / 8 = 3750 of them (the sum of the weights has the most) by
    2.1e-6, and the bound is ten of those.  Sums that are cut off lose 2^-24 to
    2^-25 of it on average each time instead, always the same way: 5e-5 to 1e-4
    for the n / 16 products of a value."""
    b = Batch([30000], 8, 1, 128, 16, "fp32", seed=27)
    fp4.write(b.cache, host(b.key), np.abs(host(b.value)), b.slots)
    ref = b.reference()[0][0]
    b.tables, b.lens = np.repeat(b.tables, 512, 0), np.repeat(b.lens, 512)
    b.query = b.query.expand(512, 8, 128).contiguous()
    got = host(Run(b)())
    assert np.max(np.abs(got - ref) / np.abs(ref)) <= 2.1e-5


@pytest.mark.parametrize("dtype,head,heads", [("bf16", 128, 4), ("bf16", 128, 8), ("bf16", 64, 16), ("bf16", 256, 8),
                                              ("fp32", 128, 4), ("fp32", 64, 8), ("fp32", 256, 8)])
def test_decode_sums_do_not_drift_with_the_length(dtype, head, heads):
    """Pairs of a million tokens, as many as warps, so that each sees about as much of one.  Every value of an element is
    the same, so that the output is that value whatever the weights are.  Off are the
    weights' roundings (bf16 2^-11, fp32 2^-22 at most), the output's (2^-8, 2^-24) and two
    sums.  bf16: chains of 2^12 tokens, 2^9 additions that may cut off 2^-23 each.  fp32:
    the same number rounded to nearest, 2^-24 / sqrt(3) in standard deviation each, of
    which ten are allowed, and the four cut-offs of a step.  Then 2^8 chains' results
    that are rounded to nearest."""
    seqs, tokens, block = 2600, 1 << 20, 256
    b = Batch([2048], heads, 1, head, block, dtype, seed=head + heads, query_std=2.0)
    value = np.resize([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -1.5], head) * (1 + np.arange(head) // 16 % 8)
    fp4.write(b.cache, host(b.key), np.broadcast_to(value, (2048, 1, head)), b.slots)
    held = fp4.read(b.cache, b.slots[:1])[1][0]
    r = Run(b)
    r.tables = r.tables.repeat(1, tokens // 2048).expand(seqs, -1).contiguous()
    r.lens = torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")
    r.query = dev(rounded(2.0 * np.random.default_rng(head).standard_normal((seqs, heads, head)), dtype))
    r.out = torch.full_like(r.query, 77.0)
    worst = np.max(np.abs(host(r()) / held - 1.0))
    deviation = 10 * 2.0 ** -24 / np.sqrt(3)
    if dtype == "bf16":
        bound = 2.0 ** -11 + 2.0 ** -8 + 2 * (2.0 ** 9 * 2.0 ** -23 + 2.0 ** 4 * deviation)
    else:
        bound = 2.0 ** -22 + 2.0 ** -24 + 4 * 2.0 ** -23 + 2 * (2.0 ** 4.5 + 2.0 ** 4) * deviation
    assert worst <= bound
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,heads", [(64, 4), (64, 16), (128, 3), (128, 8), (128, 16), (256, 4), (256, 11)])
@pytest.mark.parametrize("rise", [0.0, 120.0, -120.0])
def test_decode_long_sequences_in_a_warp(dtype, head, heads, rise):
    """Pairs of several chains of 4096 tokens and a token, more than warps, whose scores
    stay, rise (the maximum moves again and again) or fall."""
    seqs, lens = 3000, [12289, 20001, 4096, 4097]
    b = Batch([20001], heads, 1, head, 64, dtype, seed=head + heads)
    key = host(b.key)
    key[:, 0, 0] = np.linspace(0.0, 6.0, 20001)
    fp4.write(b.cache, key, host(b.value), b.slots)
    q = host(b.query).repeat(4, 0)
    q[..., 0] = rise / (6.0 * b.scale)
    b.query, b.tables, b.lens = rounded(q, dtype), b.tables.repeat(4, 0), np.array(lens, dtype=np.int32)
    ref, mass, total, reach = b.reference()
    bound = decode_bound(ref, mass, total, reach, b.lens, head, dtype)
    r = Run(b)
    r.tables, r.lens = r.tables.repeat(seqs // 4, 1), r.lens.repeat(seqs // 4)
    r.query = r.query.repeat(seqs // 4, 1, 1)
    r.out = torch.full_like(r.query, 77.0)
    got = host(r()).reshape((-1,) + ref.shape)
    assert (np.abs(got - ref) <= bound).all()


def test_decode_fp32_keeps_small_weights():
    """One token far above all others, in warps that see whole sequences: the others'
    weights are 2^-34 to 2^-33 of its, and its value is zero.  Weights are kept in steps of
    2^-24 where the largest is 2^11 at least, so each is off by half a step, 2^-36 of the
    largest, at most; relative errors of what is kept are as in decode_bound."""
    seqs, tokens, heads, head = 2600, 8193, 8, 128
    b = Batch([tokens], heads, 1, head, 256, "fp32", seed=3)
    key, value = np.full((tokens, 1, head), 0.0), np.full((tokens, 1, head), 6.0)
    key[..., 0], key[0, 0, 0], value[0] = -6.0, 6.0, 0.0
    fp4.write(b.cache, key, value, b.slots)
    gap = np.linspace(33.0, 34.0, heads)                       # powers of two between the weights
    q = np.zeros((1, heads, head))
    q[0, :, 0] = gap * np.log(2.0) / (12.0 * b.scale)
    b.query = rounded(q, "fp32")
    ref, mass, total, reach = b.reference()
    r = Run(b)
    r.tables = r.tables.expand(seqs, -1).contiguous()
    r.lens = torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")
    r.query = r.query.expand(seqs, -1, -1).contiguous()
    r.out = torch.full_like(r.query, 77.0)
    bound = decode_bound(ref, mass, 0 * total, reach, [tokens], head, "fp32") + 2.0 ** -36 * total
    assert (np.abs(host(r()) - ref) <= bound).all()


def test_decode_takes_a_long_batch_over_shared_blocks():
    """4.3 billion tokens, as many sequences on one prefix have them (2^27 units of work and more)."""
    seqs, tokens, kinds = 65535, 65536, 16
    b = Batch([tokens], 4, 1, 128, 256, seed=29)
    b.query = rounded(np.random.default_rng(30).standard_normal((kinds, 4, 128)), "bf16")
    b.tables, b.lens = np.repeat(b.tables, kinds, 0), np.repeat(b.lens, kinds)
    ref, mass, total, reach = b.reference()
    bound = decode_bound(ref, mass, total, reach, b.lens, 128, "bf16")
    r = Run(b)
    r.tables = r.tables[:1].expand(seqs, -1).contiguous()
    r.lens = r.lens[:1].expand(seqs).contiguous()
    r.query = r.query.repeat(seqs // kinds + 1, 1, 1)[:seqs].contiguous()
    r.out = torch.full_like(r.query, 77.0)
    got = host(r())
    assert pa.pa_get_device_error() == 0
    at = np.arange(seqs) % kinds
    assert (np.abs(got - ref[at]) <= bound[at]).all()


def test_decode_refuses_more_work_than_it_can_count():
    # 65535 KV heads that hold one block, read 255 times by each of 65 sequences
    heads, seqs = 65535, 65
    cache = torch.zeros((1, heads, 32, 9 * 64), dtype=torch.uint8, device="cuda")
    tables = torch.zeros((seqs + 1, 64), dtype=torch.int32, device="cuda")
    lens = torch.full((seqs + 1,), 255 * 64, dtype=torch.int32, device="cuda")
    lens[seqs] = 0
    q = torch.ones((seqs + 1, heads, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 77.0)
    ws = pa.alloc_workspace(pa.pa_decode_fp4_workspace_size(cache, heads), "cuda")
    pa.pa_decode_fp4(out, q, cache, tables, lens, 1.0, ws)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    assert not out[seqs].any()
    lens[1:] = 0                                         # the same workspace, less work
    pa.pa_decode_fp4(out, q, cache, tables, lens, 1.0, ws)
    assert pa.pa_get_device_error() == 0 and not out.any()


def test_two_graphs_share_a_workspace_and_lengths_grow():
    a = Run(Batch([70, 1, 300], 8, 2, 128, 16, seed=17))
    b = Run(Batch([9, 2000], 4, 1, 128, 16, seed=18), workspace=None)
    size = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    a(), b()
    torch.cuda.synchronize()
    graphs = []
    for r in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r()
        graphs.append(g)
    for _ in range(3):
        a.out.fill_(5), b.out.fill_(5)
        for g in graphs:
            g.replay()
        assert_decode(a.out, a.batch)
        assert_decode(b.out, b.batch)
    # the captured call on shorter and on empty sequences
    for lens in ([33, 1, 299], [0, 0, 17], [0, 0, 0]):
        a.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        a.batch.lens = np.array(lens, dtype=np.int32)
        graphs[0].replay()
        assert_decode(a.out, a.batch)


def test_two_streams_at_once():
    runs = [Run(Batch([900, 31, 40 + i], 8, 2, 64, 16, seed=19 + i)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, s in zip(runs, streams):
            r(stream=s)
    torch.cuda.synchronize()
    for r in runs:
        assert_decode(r.out, r.batch)


def test_decode_refuses_small_workspaces():
    r = Run(Batch([40], 4, 2, 64, 16))
    r.ws = r.ws[:-256]
    with pytest.raises(pa.PAError) as e:
        r()
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_decode_refuses_buffers_in_its_workspace():
    r = Run(Batch([40], 4, 2, 64, 16))
    need = pa.pa_decode_fp4_workspace_size(r.cache, 4)
    arena = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    r.ws = arena[:need]
    at = (need + 15) // 16 * 16
    for name in ("out", "query", "cache", "tables", "lens"):
        was = getattr(r, name)
        inside = arena[at - 16:at - 16 + was.nbytes] if name != "cache" else arena[:was.nbytes]
        setattr(r, name, inside.view(was.dtype).view(was.shape))
        with pytest.raises(pa.PAError) as e:
            r()
        assert e.value.status == pa.PA_ERR_INVALID_ARG, name
        setattr(r, name, was)
    r.out = arena[at:at + r.out.nbytes].view(r.out.dtype).view(r.out.shape)
    assert_decode(r(), r.batch)


def test_decode_waits_that_give_up_leave_the_workspace_usable():
    # A limit of one cycle, and more to read than L2 holds, so that most waits
    # for a copy find it not yet there and give up.
    head, hkv, block, lens = 128, 8, 16, [120_000, 5, 0, 60_001]
    counts = [-(-n // block) for n in lens]
    cache = torch.randint(0, 256, (sum(counts), hkv, block // 8, 9 * head), dtype=torch.uint8,
                          device="cuda")
    cache[..., 8 * head:] = 0x38          # every scale is one
    tables = torch.zeros((4, max(counts)), dtype=torch.int32)
    ids, at = torch.randperm(sum(counts)).int(), 0
    for r, c in enumerate(counts):
        tables[r, :c] = ids[at:at + c]
        at += c
    tables, lens = tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((4, 16, head), device="cuda").bfloat16()
    ws = pa.alloc_workspace(pa.pa_decode_fp4_workspace_size(cache, 16), "cuda")

    def call():
        out = torch.full_like(q, 5.0)
        pa.pa_decode_fp4(out, q, cache, tables, lens, head ** -0.5, ws)
        return out

    first = call()
    assert pa.pa_get_device_error() == 0 and not (first == 5.0).all(-1).any()
    pa.pa_set_decode_wait_limit(1)
    try:
        call()
        assert pa.pa_get_device_error() == pa.PA_DEVERR_TIMEOUT
    finally:
        pa.pa_set_decode_wait_limit(0)
    for _ in range(2):
        assert torch.equal(call(), first)
    assert pa.pa_get_device_error() == 0


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

class Tables:
    """A step of the tables on the device and in the oracle."""

    def __init__(self, lens, new, block, width=None, ring=True, spare=5, seed=0, most=None):
        rng = np.random.default_rng(seed)
        lens, new = np.asarray(lens, dtype=np.int64), np.asarray(new, dtype=np.int64)
        total = np.maximum(-(-(lens + np.maximum(new, 0)) // block), 0)
        self.block, self.blocks = block, int(total.sum()) + spare
        have = -(-lens // block) if ring else total
        width = int(max(1, total.max(initial=1))) if width is None else width
        perm = rng.permutation(self.blocks).astype(np.int32)
        self.tables = np.full((len(lens), width), -7, dtype=np.int32)
        at = 0
        for r, c in enumerate(have):
            self.tables[r, :c] = perm[at:at + c]
            at += c
        self.lens, self.new = lens.astype(np.int32), new.astype(np.int32)
        self.ring = self.state = None
        if ring:
            front = int(rng.integers(0, self.blocks - at))
            self.ring = np.roll(perm[at:], front)
            self.state = np.array([front, self.blocks - at], dtype=np.int32)
        self.most = int(max(new.sum(), 0)) + 3 if most is None else most

    def check(self, in_place=False, error=0):
        t, ln, new = dev(self.tables), dev(self.lens), dev(self.new)
        ring = None if self.ring is None else dev(self.ring)
        state = None if self.state is None else dev(self.state)
        n = len(self.lens)
        slots = torch.full((self.most,), 99, dtype=torch.int64, device="cuda")
        pos = torch.full((self.most,), 99, dtype=torch.int32, device="cuda")
        starts = torch.full((n + 1,), 99, dtype=torch.int32, device="cuda")
        lo = ln if in_place else torch.full_like(ln, 99)
        so = state if in_place or state is None else torch.full_like(state, 99)
        pa.pa_extend_tables(t, ln, new, self.block, self.blocks, slots, pos, starts,
                            seq_lens_out=lo, free_blocks=ring, free_state=state, free_state_out=so)
        assert pa.pa_get_device_error() == error
        want = fp4.extend_tables(self.tables, self.lens, self.new, self.block, self.blocks,
                                 self.most, self.ring, self.state)
        assert want[6] == (error in (pa.PA_DEVERR_SEQ_LEN, pa.PA_DEVERR_BLOCKS))
        for name, got, ref in (("tables", t, want[0]), ("lens", lo, want[1]), ("slots", slots, want[3]),
                               ("positions", pos, want[4]), ("starts", starts, want[5])):
            assert np.array_equal(host(got), ref), name
        if state is not None:
            assert host(so).tolist() == list(want[2])
        if not in_place:
            assert np.array_equal(host(ln), self.lens)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ring", [True, False])
@pytest.mark.parametrize("block", [1, 8, 16, 256])
def test_tables(block, ring, in_place):
    rng = np.random.default_rng(block)
    Tables([0, 1, 15, 16, 17, 255, 256, 40], [1, 0, 1, 1, 300, 1, 1, 0], block, ring=ring).check(in_place)
    Tables([5], [1], block, ring=ring).check(in_place)
    Tables([0], [0], block, ring=ring).check(in_place)
    Tables(rng.integers(0, 200, 333), rng.integers(0, 40, 333), block, ring=ring).check(in_place)
    Tables(rng.integers(0, 50, 700), np.ones(700, int), block, ring=ring).check(in_place)


def test_tables_many_requests_and_tokens():
    rng = np.random.default_rng(3)
    Tables(rng.integers(0, 30, 8192), rng.integers(0, 3, 8192), 16).check(True)
    Tables(rng.integers(0, 3, 2049), np.where(np.arange(2049) == 1000, 50_001, 0), 8).check()
    Tables([3, 9], [70_000, 1], 16, most=90_000).check()


def test_tables_most_tokens():
    n, block = (1 << 26) - 1, 256
    blocks = (1 << 18) + 3
    ring = torch.randperm(blocks, device="cuda").int()
    tables = torch.full((2, 1 << 18), -7, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    new = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    state = torch.tensor([1000, blocks], dtype=torch.int32, device="cuda")
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    pos = torch.empty(n, dtype=torch.int32, device="cuda")
    for in_place in (False, True):
        lo, so = (lens, state) if in_place else (torch.empty_like(lens), torch.empty_like(state))
        slots.fill_(99), pos.fill_(99)
        pa.pa_extend_tables(tables, lens, new, block, blocks, slots, pos, seq_lens_out=lo,
                            free_blocks=ring, free_state=state, free_state_out=so)
        at = torch.arange(n, device="cuda")
        assert torch.equal(pos, at.int())
        ids = torch.roll(ring, -1000)[:1 << 18]
        assert torch.equal(tables[1], ids) and (tables[0] == -7).all()
        assert torch.equal(slots, ids.long()[at >> 8] * 256 + (at & 255))
        assert lo.tolist() == [0, n] and so.tolist() == [1000 - 3, 3]
        assert pa.pa_get_device_error() == 0


def test_calls_take_numpy_scalars():
    b = Batch([20, 3], 4, 2, 64, 8, seed=28, key_scale=2.0, value_scale=0.5)
    r = Run(b)
    r.ws = pa.alloc_workspace(pa.pa_decode_fp4_workspace_size(r.cache, np.int64(4)), "cuda")
    b.scale, b.key_scale, b.value_scale = np.float32(b.scale), np.float32(2), np.float32(0.5)
    assert_decode(r(), b)
    ko = torch.empty((1, 2, 64), device="cuda")
    vo = torch.empty_like(ko)
    one = torch.zeros(1, dtype=torch.int64, device="cuda")
    pa.pa_reshape_and_cache_fp4(r.cache, ko.fill_(12), vo.fill_(3), one, np.float32(2), np.float32(0.5))
    pa.pa_gather_cache_fp4(ko, vo, r.cache, one, np.float32(2), np.float32(0.5))
    assert (ko == 12).all() and (vo == 3).all()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_extend_tables(lens.view(1, 1).clone(), lens, lens + 1, np.int64(8), np.int64(5), one)
    assert one.tolist() == [0] and lens.tolist() == [1]


def test_tables_refuse_whole_steps():
    for kw in (dict(lens=[3, 5], new=[1, -1]), dict(lens=[3, -5], new=[1, 1]),
               dict(lens=[3, 30], new=[14, 3], width=2),
               dict(lens=[3, 30], new=[14, 4], most=17),
               dict(lens=[3, 3, 3], new=[(1 << 31) - 1, (1 << 31) - 1, 5], width=4, most=8, spare=9)):
        if max(kw["new"]) > 1000:
            t = Tables([3, 3, 3], [1, 1, 5], 16, width=4, most=8)
            t.new = np.array(kw["new"], dtype=np.int32)
            # the oracle walks tokens: it meets the end of the row
            t.check(error=pa.PA_DEVERR_SEQ_LEN)
            continue
        for in_place in (False, True):
            Tables(block=16, **kw).check(in_place, error=pa.PA_DEVERR_SEQ_LEN)
    t = Tables([3, 16, 40], [1, 1, 100], 16, spare=3)
    t.state[1] = 6                       # seven are needed
    t.check(error=pa.PA_DEVERR_BLOCKS)
    t.check(True, error=pa.PA_DEVERR_BLOCKS)
    t.state[1] = 7
    t.check()


def test_tables_bad_ids_lose_their_tokens():
    t = Tables([16, 20], [2, 1], 16)
    t.ring[:] = t.blocks                 # past the pool
    t.check(error=pa.PA_DEVERR_BLOCK_ID)
    t = Tables([16, 20], [2, 1], 16, ring=False)
    t.tables[1, 1] = -1
    t.check(error=pa.PA_DEVERR_BLOCK_ID)


def test_tables_without_requests():
    slots = torch.full((5,), 4, dtype=torch.int64, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    starts = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    pa.pa_extend_tables(torch.empty((0, 3), dtype=torch.int32, device="cuda"), e, e, 16, 4, slots,
                        token_starts=starts)
    assert (slots == -1).all() and (starts == 0).all()


# ---------------------------------------------------------------------------
# the step
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,heads,hkv,head,block", [("bf16", 8, 2, 128, 16), ("bf16", 5, 5, 64, 8),
                                                        ("fp32", 6, 2, 256, 16)])
def test_captured_step_serves_growing_sequences(dtype, heads, hkv, head, block):
    """tables -> write -> decode captured once, replayed for every step: the
    device's tables agree with the host pool's, the attention with the oracle
    fed the same tokens."""
    rng = np.random.default_rng(head)
    prompts = [3, block, 0, 4 * block - 1]
    blocks, width, steps = 40, 10, 2 * block + 3
    pool = pa.Pool(blocks, block, free_order=rng.permutation(blocks))
    seqs = [pool.add_seq(n) for n in prompts]
    tables, lens = pool.fill_tables(seqs, width)
    ring = dev(np.array(pool.free_queue(), dtype=np.int32))
    state = torch.tensor([0, pool.num_free()], dtype=torch.int32, device="cuda")
    tables, lens = tables.cuda(), lens.cuda()
    cache = torch.randint(0, 256, (blocks, hkv, block // 8, 9 * head), dtype=torch.uint8, device="cuda")
    # prompts
    n = sum(prompts)
    pk = rounded(rng.standard_normal((n, hkv, head)), dtype)
    pv = rounded(rng.standard_normal((n, hkv, head)), dtype)
    slots0 = torch.full((n + 2,), -1, dtype=torch.int64, device="cuda")
    pa.pa_extend_tables(tables, torch.zeros_like(lens), lens, block, blocks, slots0,
                        seq_lens_out=torch.empty_like(lens))
    pa.pa_reshape_and_cache_fp4(cache, dev(pk), dev(pv), slots0[:n])
    ref = cache.cpu().numpy().copy()
    fp4.write(ref, host(pk), host(pv), host(slots0[:n]))

    s = len(prompts)
    new = torch.ones(s, dtype=torch.int32, device="cuda")
    slots = torch.empty(s, dtype=torch.int64, device="cuda")
    qkv = torch.zeros((s, (heads + 2 * hkv) * head), dtype=TORCH[dtype], device="cuda")
    q, k, v = qkv.split([heads * head, hkv * head, hkv * head], dim=1)
    q, k, v = q.unflatten(1, (heads, head)), k.unflatten(1, (hkv, head)), v.unflatten(1, (hkv, head))
    out = torch.empty((s, heads, head), dtype=TORCH[dtype], device="cuda")
    ws = pa.alloc_workspace(pa.pa_decode_fp4_workspace_size(cache, heads), "cuda")

    def step():
        pa.pa_extend_tables(tables, lens, new, block, blocks, slots, free_blocks=ring, free_state=state)
        pa.pa_reshape_and_cache_fp4(cache, k, v, slots)
        pa.pa_decode_fp4(out, q, cache, tables, lens, head ** -0.5, ws)

    saved = [t.clone() for t in (tables, lens, state, cache)]
    step()                               # once outside, then put everything back
    torch.cuda.synchronize()
    for t, was in zip((tables, lens, state, cache), saved):
        t.copy_(was)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(steps):
        x = rounded(rng.standard_normal(tuple(qkv.shape)), dtype)
        qkv.copy_(x)
        g.replay()
        want_slots, pairs = pool.append_tokens(seqs)
        assert pairs.numel() == 0 and torch.equal(slots.cpu(), want_slots)
        fp4.write(ref, host(k), host(v), want_slots.numpy())
        if i % 5 and i != steps - 1:
            continue
        b = Batch([1], heads, hkv, head, block, dtype)  # a shell for the bound
        b.cache, b.query = ref, q.detach().cpu()
        bt, ln = pool.fill_tables(seqs, width)
        b.tables, b.lens = bt.numpy(), ln.numpy()
        assert np.array_equal(host(lens), b.lens)
        assert_decode(out, b, "step %d" % i)
    assert host(state)[1] == pool.num_free() and pa.pa_get_device_error() == 0


@pytest.mark.parametrize("in_place", [True, False])
def test_prompt_steps_in_a_row_see_what_the_step_before_wrote(in_place):
    """Steps of thousands of tokens (tables by several CTAs) captured one behind another, so
    that each launch starts while the ones before still run; every step's tables, slots and
    attention."""
    rng = np.random.default_rng(33)
    n, steps, most, block, blocks, width = 24, 6, 5000, 8, 4000, 320
    heads, hkv, head = 4, 1, 64
    i32 = lambda a: dev(np.asarray(a, dtype=np.int32))
    new = rng.integers(0, 400, (steps, n))
    new[:, ::5] = 1
    ring = rng.permutation(blocks)
    cache = torch.randint(0, 256, (blocks, hkv, 1, 9 * head), dtype=torch.uint8, device="cuda")
    first = cache.cpu().numpy().copy()
    k, v = (dev(rounded(rng.standard_normal((steps, most, hkv, head)), "bf16")) for _ in range(2))
    q = dev(rounded(rng.standard_normal((steps, n, heads, head)), "bf16"))
    out = torch.empty_like(q)
    tables = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    lens = [torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(steps + 1)]
    state = [i32([7, blocks]) for _ in range(steps + 1)]
    slots = torch.empty((steps, most), dtype=torch.int64, device="cuda")
    free, news = i32(ring), i32(new)
    ws = pa.alloc_workspace(pa.pa_decode_fp4_workspace_size(cache, heads), "cuda")
    at = lambda i: 0 if in_place else i

    def run():
        for i in range(steps):
            pa.pa_extend_tables(tables, lens[at(i)], news[i], block, blocks, slots[i], free_blocks=free,
                                free_state=state[at(i)], seq_lens_out=lens[at(i + 1)],
                                free_state_out=state[at(i + 1)])
            pa.pa_reshape_and_cache_fp4(cache, k[i], v[i], slots[i])
            pa.pa_decode_fp4(out[i], q[i], cache, tables, lens[at(i + 1)], head ** -0.5, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    ref, t, ln, st = first.copy(), np.full((n, width), -1), np.zeros(n, int), [7, blocks]
    want = []
    b = Batch([1], heads, hkv, head, block)  # a shell for the bound
    for i in range(steps):
        t, ln, st, sl, _, _, refused = fp4.extend_tables(t, ln, new[i], block, blocks, most, ring, st)
        assert not refused
        fp4.write(ref, host(k[i]), host(v[i]), sl)
        r = fp4.decode(host(q[i]), ref, t, ln, b.scale)
        want.append((sl, r[0], decode_bound(*r, ln, head, "bf16")))
    for _ in range(5):
        cache.copy_(dev(first)), tables.fill_(-1), lens[0].zero_(), state[0].copy_(i32([7, blocks]))
        g.replay()
        torch.cuda.synchronize()
        for i, (sl, r, bound) in enumerate(want):
            assert np.array_equal(host(slots[i]), sl), i
            assert (np.abs(host(out[i]) - r) <= bound).all(), i
        assert np.array_equal(host(lens[at(steps)]), ln) and host(state[at(steps)]).tolist() == list(st)
        assert np.array_equal(host(tables), t)
    assert pa.pa_get_device_error() == 0


FIRST_CALLS = """
import torch
import paged_kv_cache_78_gb300 as pa
t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache = pa.alloc_fp4_cache(6, 8, 1, 64)
kv = torch.full((2, 1, 64), 6.0, device="cuda")
out, back = torch.empty((2, 1, 64), device="cuda"), torch.empty((2, 2, 1, 64), device="cuda")
tables, lens, new, state = t(1, 2, 3, 4).view(2, 2), t(0, 7), t(1, 1), t(0, 2)
slots = torch.empty(2, dtype=torch.int64, device="cuda")
ws = pa.alloc_workspace(pa.pa_decode_fp4_workspace_size(cache, 1), "cuda")
ring = t(5, 0)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pa.pa_extend_tables(tables, lens, new, 8, 6, slots, free_blocks=ring, free_state=state)
    pa.pa_reshape_and_cache_fp4(cache, kv, kv, slots)
    pa.pa_gather_cache_fp4(back[0], back[1], cache, slots)
    pa.pa_decode_fp4(out, kv, cache, tables, lens, 1.0, ws)
g.replay()
assert slots.tolist() == [40, 31] and (back == 6).all() and state.tolist() == [1, 1]
assert (out - 6).abs().max() < 1e-5
print("captured")
"""


def test_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True,
                       timeout=280)
    assert r.returncode == 0 and r.stdout.split()[-1] == "captured", r.stderr
