"""The 8-bit pool on the GPU against the binary64 oracle: quantising write and read-back
(exact), block copies (exact), decode attention and the blocks' weights (within bounds
derived from the roundings)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_78_gb300 as pa
from int8_util import (TORCH, Batch, assert_decode, assert_weights, decode_bound, host, rounded, score_bound,
                       weights_bound)
from oracle import int8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    pa.pa_get_device_error()
    yield


def dev(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).cuda()


def same(a, b):
    return np.array_equal(np.asarray(a, dtype=np.float64), b, equal_nan=True)


def held(cache, slots, dtype):
    """What a read-back gives: code * scale in fp32, then in the type."""
    out = []
    for x in int8.read(cache, slots):
        with np.errstate(over="ignore", invalid="ignore"):
            out.append(host(torch.from_numpy(x.astype(np.float32)).to(TORCH[dtype])))
    return out


def assert_pool(got, want, slots, what=""):
    """Codes and every tile's scales of the blocks that the slots name, and all bytes of others."""
    bs = want.shape[2] * 8
    mine = np.unique(np.asarray(slots) // bs)
    others = np.setdiff1d(np.arange(len(want)), mine)
    assert np.array_equal(got[others], want[others]), what
    for b in mine:
        live = np.unique(np.asarray(slots)[np.asarray(slots) // bs == b] % bs)
        for side in range(2):
            assert same(int8.block_scales(got, b, side), int8.block_scales(want, b, side)), (what, b)
            assert np.array_equal(int8.block_codes(got, b, side)[:, live],
                                  int8.block_codes(want, b, side)[:, live]), (what, b)
        assert np.array_equal(got[b, :, :, 8:16], want[b, :, :, 8:16]), what


# ---------------------------------------------------------------------------
# write and read-back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,hkv,block,lens", [
    (64, 1, 8, [1]), (64, 3, 16, [77, 5]), (128, 8, 16, [130, 16, 33]), (128, 2, 256, [300, 700]),
    (256, 5, 32, [41]), (64, 1, 8, [1001]), (64, 40, 16, [65]), (128, 1, 16, [3, 3, 3, 3]),
    (256, 1, 8, [9]), (256, 2, 128, [500, 1]), (128, 2, 16, [4000, 3333])])
def test_prompts(dtype, head, hkv, block, lens):
    """Whole sequences in one call, rows in any order inside a block, into a pool of random bytes;
    then both are read back."""
    rng = np.random.default_rng(head + sum(lens))
    nb = sum(-(-n // block) for n in lens) + 3
    cache = rng.integers(-128, 128, (nb, hkv, block // 8, 16 * (head + 1)), dtype=np.int8)
    ids, slots = rng.permutation(nb), []
    for n in lens:
        for b in range(-(-n // block)):
            off = rng.permutation(min(block, n - b * block))
            slots.append(ids[0] * block + off)
            ids = ids[1:]
    slots = np.concatenate(slots).astype(np.int64)
    n = len(slots)
    k = rounded(4 * rng.standard_normal((n, hkv, head)) * np.exp(rng.standard_normal((n, hkv, 1))), dtype)
    v = rounded(0.1 * rng.standard_normal((n, hkv, head)), dtype)
    d = dev(cache)
    pa.pa_reshape_and_cache_int8(d, dev(k), dev(v), dev(slots))
    want = cache.copy()
    int8.write(want, host(k), host(v), slots)
    assert_pool(d.cpu().numpy(), want, slots)
    again = np.concatenate([slots, slots[:3]])            # the read-back takes slots repeated
    ko = torch.empty((len(again), hkv, head), dtype=TORCH[dtype], device="cuda")
    vo = torch.empty_like(ko)
    pa.pa_gather_cache_int8(ko, vo, d, dev(again))
    rk, rv = held(want, again, dtype)
    assert same(host(ko), rk) and same(host(vo), rv)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,hkv,block,seqs", [(64, 2, 16, 64), (128, 3, 8, 5), (256, 1, 256, 3), (128, 8, 32, 300)])
def test_tokens_appended_one_by_one(dtype, head, hkv, block, seqs):
    """Steps of one token for each sequence: scales stay, grow (what the blocks hold is rounded
    again) and begin anew."""
    rng = np.random.default_rng(head)
    steps = min(2 * block + 1, 40)
    need = -(-(steps + block) // block)
    cache = rng.integers(-128, 128, (seqs * need, hkv, block // 8, 16 * (head + 1)), dtype=np.int8)
    tables = rng.permutation(seqs * need).reshape(seqs, need)
    start = rng.integers(0, block, seqs)
    slots = lambda i: tables[np.arange(seqs), (start + i) // block] * block + (start + i) % block
    d, want = dev(cache), cache.copy()
    every = []
    # what stands before the first step, so that scales are numbers
    first = np.concatenate([tables[r, 0] * block + np.arange(n) for r, n in enumerate(start)] or [[]]).astype(np.int64)
    x = rounded(rng.standard_normal((len(first), hkv, head)), dtype)
    pa.pa_reshape_and_cache_int8(d, dev(x), dev(-x), dev(first))
    int8.write(want, host(x), host(-x), first)
    for i in range(steps):
        s = slots(i)
        size = np.exp(rng.standard_normal((seqs, hkv, 1)))
        k, v = (rounded(size * rng.standard_normal((seqs, hkv, head)), dtype) for _ in range(2))
        pa.pa_reshape_and_cache_int8(d, dev(k), dev(v), dev(s))
        int8.write(want, host(k), host(v), s)
        every.append(s)
    assert_pool(d.cpu().numpy(), want, np.concatenate(every + [first]))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_chunks_that_continue_blocks(dtype):
    """Prompts in chunks of every length about a block's and a window's, many in a call."""
    rng = np.random.default_rng(3)
    block, hkv, head = 16, 2, 128
    lens = np.zeros(40, dtype=int)
    tables = rng.permutation(40 * 12).reshape(40, 12)
    cache = rng.integers(-128, 128, (480, hkv, 2, 16 * (head + 1)), dtype=np.int8)
    d, want = dev(cache), cache.copy()
    every = []
    for _ in range(4):
        new = rng.choice([0, 1, 2, 15, 16, 17, 31, 33, 40], 40)
        at = [tables[r, (lens[r] + np.arange(n)) // block] * block + (lens[r] + np.arange(n)) % block
              for r, n in enumerate(new)]
        s = np.concatenate(at).astype(np.int64)
        k, v = (rounded(np.exp(rng.standard_normal((len(s), 1, 1))) * rng.standard_normal((len(s), hkv, head)), dtype)
                for _ in range(2))
        pa.pa_reshape_and_cache_int8(d, dev(k), dev(v), dev(s))
        int8.write(want, host(k), host(v), s)
        lens += new
        every.append(s)
    assert_pool(d.cpu().numpy(), want, np.concatenate(every))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,hkv,block,blocks", [(64, 5, 8, 2300), (64, 3, 256, 60), (128, 2, 128, 90), (256, 1, 64, 100)])
def test_many_runs_of_any_length(dtype, head, hkv, block, blocks):
    """Blocks that begin with any number of tokens, many of them whole, one or none, in any order
    with padding between them; then what is left of some, larger in every other one, so that
    their scales grow.  More runs, heads and sides than the GPU takes at once."""
    rng = np.random.default_rng(head + block)
    cache = rng.integers(-128, 128, (blocks, hkv, block // 8, 16 * (head + 1)), dtype=np.int8)
    first = np.where(rng.random(blocks) < 0.5, block, rng.integers(0, block + 1, blocks))
    first = np.where(rng.random(blocks) < 0.1, 1, first)
    second = np.where(first > 0, np.minimum(block, first + rng.integers(0, block + 1, blocks)), 0)
    d, want = dev(cache), cache.copy()
    for begin, end in ((np.zeros(blocks, int), first), (first, second)):
        slots = []
        for b in rng.permutation(blocks):
            slots.append(b * block + begin[b] + rng.permutation(end[b] - begin[b]))
            slots.append(np.full(rng.integers(0, 3) * (rng.random() < 0.3), -1))
        slots = np.concatenate(slots).astype(np.int64)
        n = len(slots)
        size = np.where(slots // block % 2 == 0, 3.0, 1.0)[:, None, None] if begin.any() else 1.0
        k = rounded(size * rng.standard_normal((n, hkv, head)), dtype)
        v = rounded(size * rng.standard_normal((n, hkv, head)), dtype)
        pa.pa_reshape_and_cache_int8(d, dev(k), dev(v), dev(slots))
        int8.write(want, host(k), host(v), slots)
    live = np.concatenate([b * block + np.arange(n) for b, n in enumerate(second)])
    assert_pool(d.cpu().numpy(), want, live)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_codes_round_on_the_exact_quotients(dtype):
    """Every border between two codes times scales of many mantissas, the nearest number of the type
    and its neighbours; a maximum of 127 times the scale fixes it."""
    rows = []
    rng = np.random.default_rng(4)
    for s in np.concatenate([2.0 ** np.array([-120.0, -20, 0, 100]), rng.uniform(1, 2, 60), rng.uniform(1, 2, 4) * 1e-36]):
        top = float(rounded(np.array([127 * s]), dtype).double()[0])
        scale = float(np.float32(top / 127))
        border = rounded((rng.permutation(127)[:20] + 0.5) * scale, dtype)
        for x in (border, torch.nextafter(border, torch.full_like(border, float("inf"))),
                  torch.nextafter(border, torch.zeros_like(border))):
            rows.append(np.concatenate([[top], host(x), -host(x), np.zeros(64 - 41)]))
    x = np.array(rows)[:, None, :]
    key = rounded(x, dtype)
    n = len(rows)
    cache = torch.zeros((n, 1, 1, 16 * 65), dtype=torch.int8, device="cuda")
    slots = 8 * np.arange(n)                                 # each begins a block
    pa.pa_reshape_and_cache_int8(cache, dev(key), dev(-key), dev(slots))
    want = np.zeros(tuple(cache.shape), dtype=np.int8)
    int8.write(want, host(key), host(-key), slots)
    assert_pool(cache.cpu().numpy(), want, slots)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_growing_scales_round_codes_on_the_exact_quotients(dtype):
    """A block of all codes whose scale then grows by ratios with ties and near them."""
    rng = np.random.default_rng(5)
    codes = np.arange(-127, 128)
    ratio = np.concatenate([[2.0, 4.0, 1.0, 254.0 / 127, 1.5, 3.0, 1 + 2.0 ** -7, 1e30, 128.0], rng.uniform(1, 4, 30)])
    base = np.concatenate([[1.0, 2.0 ** -100, 2.0 ** 60], rng.uniform(1, 2, len(ratio) - 3)])
    n = len(ratio)
    block = np.zeros((n, 8, 1, 64))
    block.reshape(n, 512)[:, :255] = codes
    block *= base[:, None, None, None]
    first = rounded(block.reshape(n * 8, 1, 64), dtype)
    cache = torch.zeros((n, 1, 1, 16 * 65), dtype=torch.int8, device="cuda")
    want = np.zeros(tuple(cache.shape), dtype=np.int8)
    more = np.zeros((n, 1, 64))
    more[:, 0, 3] = 127 * base * ratio
    second = rounded(more, dtype)
    every, last = np.arange(8 * n), 8 * np.arange(n) + 7
    for x, s in ((first, every), (second, last)):
        pa.pa_reshape_and_cache_int8(cache, dev(x), dev(-x), dev(s))
        int8.write(want, host(x), host(-x), s)
    assert_pool(cache.cpu().numpy(), want, every)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_special_values(dtype):
    rng = np.random.default_rng(7)
    x = rng.standard_normal((8, 2, 64))
    x[0, 0, 3] = np.nan
    x[1, 1, 17] = np.inf
    x[2, 0, 40] = -np.inf
    x[3] = 0.0
    x[4] = 1e-39 * rng.standard_normal((2, 64))            # below the normal numbers
    x[5] = 3e38 * np.sign(rng.standard_normal((2, 64)))
    x[6] = 2.0 ** -149
    x[7, :, ::2] = 2.0 ** -133
    t = rounded(x, dtype)
    cache = torch.randint(-128, 128, (8, 2, 1, 16 * 65), dtype=torch.int8, device="cuda")
    want = cache.cpu().numpy()
    for off in range(2):                                   # begins; goes on, the sides exchanged
        y = t if off == 0 else t.flip(0)
        slots = 8 * np.arange(8) + off
        pa.pa_reshape_and_cache_int8(cache, dev(y), dev(y.flip(1)), dev(slots))
        int8.write(want, host(y), host(y.flip(1)), slots)
    every = np.arange(16) // 2 * 8 + np.arange(16) % 2
    assert_pool(cache.cpu().numpy(), want, every)
    ko = torch.empty((16, 2, 64), dtype=TORCH[dtype], device="cuda")
    vo = torch.empty_like(ko)
    pa.pa_gather_cache_int8(ko, vo, cache, dev(every))
    rk, rv = held(want, every, dtype)
    assert same(host(ko), rk) and same(host(vo), rv)
    assert np.isnan(rk).any() and np.isfinite(rk).any()


def test_padding_and_slots_outside_the_pool():
    rng = np.random.default_rng(8)
    cache = rng.integers(-128, 128, (3, 2, 2, 16 * 65), dtype=np.int8)
    k = rounded(rng.standard_normal((6, 2, 64)), "bf16")
    slots = np.array([16, -1, 48, 32, 1 << 40, -(1 << 40)], dtype=np.int64)
    d = dev(cache)
    pa.pa_reshape_and_cache_int8(d, dev(k), dev(k), dev(slots))
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SLOT
    want = cache.copy()
    int8.write(want, host(k), host(k), slots)
    assert_pool(d.cpu().numpy(), want, [16, 32])
    ko = torch.full((6, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 8.0)
    pa.pa_gather_cache_int8(ko, vo, d, dev(slots))
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SLOT
    rk, rv = held(want, slots[[0, 3]], "bf16")
    assert same(host(ko)[[0, 3]], rk) and same(host(vo)[[0, 3]], rv)
    assert (host(ko)[[1, 2, 4, 5]] == 9).all() and (host(vo)[[1, 2, 4, 5]] == 8).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,hkv", [(64, 3), (128, 2), (256, 1)])
def test_rows_that_lie_apart_and_off_32_byte_boundaries(dtype, head, hkv):
    rng = np.random.default_rng(head)
    n, half = 37, 8 if dtype == "bf16" else 4                  # elements of 16 bytes
    slots = np.arange(5, 5 + n)
    for off, odd in ((half, 0), (0, half), (half, 3 * half)):
        stride = hkv * head + odd
        key, value = (dev(rounded(rng.standard_normal(n * stride + half), dtype))
                      .as_strided((n, hkv, head), (stride, head, 1), off) for _ in range(2))
        cache = torch.zeros((3, hkv, 2, 16 * (head + 1)), dtype=torch.int8, device="cuda")
        want = np.zeros(tuple(cache.shape), dtype=np.int8)
        pa.pa_reshape_and_cache_int8(cache, key, value, dev(slots))
        int8.write(want, host(key), host(value), slots)
        assert_pool(cache.cpu().numpy(), want, slots)
        k, v = held(want, slots, dtype)
        size = n * hkv * head
        for at, bt in ((half, half), (0, half), (half, 0)):    # one of the outputs, or both
            flat = torch.full((2, size + 2 * half), 7.0, dtype=TORCH[dtype], device="cuda")
            ko, vo = flat[0, at:at + size], flat[1, bt:bt + size]
            pa.pa_gather_cache_int8(ko.view(n, hkv, head), vo.view(n, hkv, head), cache, dev(slots))
            assert same(host(ko).reshape(k.shape), k) and same(host(vo).reshape(v.shape), v)
            for row, x in ((flat[0], at), (flat[1], bt)):
                assert (row[:x] == 7).all() and (row[x + size:] == 7).all()
    if hkv > 1:  # heads that do not lie behind one another (one head always does)
        with pytest.raises(ValueError):
            pa.pa_reshape_and_cache_int8(cache, key.transpose(1, 2).contiguous().transpose(1, 2), value, dev(slots))
    with pytest.raises(pa.PAError):  # rows that start off a 16-byte boundary
        x = torch.zeros(n * hkv * head + 1, dtype=TORCH[dtype], device="cuda")[1:].view(n, hkv, head)
        pa.pa_reshape_and_cache_int8(cache, x, value, dev(slots))


def test_no_tokens():
    c = pa.alloc_int8_cache(2, 8, 2, 64)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    pa.pa_reshape_and_cache_int8(c, k, k, s)
    pa.pa_gather_cache_int8(k, k, c, s)


@pytest.mark.parametrize("head,hkv,block", [(64, 1, 8), (128, 3, 16), (256, 2, 64)])
def test_block_copies(head, hkv, block):
    rng = np.random.default_rng(head)
    a = rng.integers(-128, 128, (9, hkv, block // 8, 16 * (head + 1)), dtype=np.int8)
    d = dev(a)
    pa.pa_copy_blocks(d, torch.tensor([[0, 7], [3, 1], [8, 2]], device="cuda"))
    want = a.copy()
    want[[7, 1, 2]] = a[[0, 3, 8]]
    assert np.array_equal(d.cpu().numpy(), want)
    cpu = torch.zeros((4, hkv, block // 8, 16 * (head + 1)), dtype=torch.int8).pin_memory()
    pa.pa_swap_blocks(cpu, d, torch.tensor([[7, 3], [4, 0]], device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(cpu.numpy()[[3, 0]], want[[7, 4]]) and not cpu[1:3].any()
    pa.pa_swap_blocks(d, cpu, torch.tensor([[3, 5]], device="cuda"))
    want[5] = want[7]
    assert np.array_equal(d.cpu().numpy(), want)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

class Run:
    """A batch on the device and its decode; with `decay` the blocks' weights too."""

    def __init__(self, batch, workspace=None, decay=None):
        b = self.batch = batch
        self.cache, self.query = dev(b.cache), dev(b.query)
        self.tables, self.lens = dev(b.tables), dev(b.lens)
        self.out = torch.full_like(self.query, 77.0)
        self.decay, self.old, self.new = decay, dev(b.old), torch.full(b.old.shape, 5.0, device="cuda")
        self.ws = workspace
        if workspace is None:
            self.ws = pa.alloc_workspace(
                pa.pa_decode_int8_workspace_size(self.cache, b.query.shape[1],
                                                 None if decay is None else self.tables), "cuda")

    def __call__(self, stream=None):
        b = self.batch
        keep = {} if self.decay is None else dict(block_weights=self.old, block_weights_out=self.new,
                                                  decay=self.decay)
        pa.pa_decode_int8(self.out, self.query, self.cache, self.tables, self.lens, b.scale, self.ws,
                          stream=stream, **keep)
        return self.out

    def check(self, what=""):
        """One call with everything against the oracle."""
        ref = self.batch.reference()
        assert_decode(self(), self.batch, what, ref)
        if self.decay is not None:
            assert_weights(self.new, self.batch, self.batch.old, self.decay, np.full(self.batch.old.shape, 5.0),
                           what, ref)


EDGES = [0, 1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 0, 255, 257, 500]


@pytest.mark.parametrize("decay", [None, 0.75])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,block", [(64, 8), (64, 16), (128, 8), (128, 16), (128, 64), (256, 8), (256, 16),
                                        (256, 256), (64, 128), (128, 32)])
def test_decode_edge_lengths(dtype, head, block, decay):
    Run(Batch(EDGES, 8, 2, head, block, dtype, seed=head + block), decay=decay).check()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("group", list(range(1, 17)))
@pytest.mark.parametrize("head", [64, 128, 256])
def test_decode_groups(head, group):
    hkv = 1 + group % 3
    for dtype in ("bf16", "fp32"):
        for block in (16, 8):
            Run(Batch([3, 100, 45], hkv * group, hkv, head, block, dtype, seed=group), decay=1.0).check(dtype)


@pytest.mark.parametrize("decay", [None, 1.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,heads,hkv,head,block", [
    ([4096], 8, 1, 128, 16),              # one pair over many CTAs
    ([5000, 1, 0, 3001], 4, 4, 64, 16),
    ([20001], 16, 1, 64, 32),
    ([2500, 777], 12, 2, 256, 8),
    ([9000], 16, 1, 128, 16),
    ([300] * 40, 40, 40, 128, 16),        # more pairs than CTAs
    (list(range(0, 900, 7)), 7, 1, 128, 8),
])
def test_decode_larger(lens, heads, hkv, head, block, dtype, decay):
    r = Run(Batch(lens, heads, hkv, head, block, dtype, seed=len(lens)), decay=decay)
    r.check()
    # again on the same workspace, and the same bits
    first, weights = r.out.clone(), r.new.clone()
    r.out.fill_(55.0)
    assert torch.equal(r(), first) and torch.equal(r.new, weights)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_peaked_and_scaled(dtype):
    # large scores (weights close to 0 and 1), keys, values and queries of other sizes
    shape = dict(heads=6, kv_heads=2, head=128, block=16, dtype=dtype)
    rng = np.random.default_rng(5)
    n = 50 + 700 + 33
    kv = lambda size: size * rng.standard_normal((n, 2, 128))
    Run(Batch([50, 700, 33], seed=5, key=kv(4.0), value=kv(2.0 ** -6), query_std=30.0, **shape), decay=0.5).check()
    Run(Batch([50, 700, 33], seed=6, query_std=2.0 ** -40, **shape), decay=0.5).check()
    Run(Batch([50, 700, 33], seed=7, key=kv(2.0 ** -30), query_std=2.0 ** 30, **shape), decay=0.5).check()
    Run(Batch([50, 700, 33], seed=7, value=kv(2.0 ** -100), **shape), decay=0.5).check()
    Run(Batch([50, 700, 33], seed=7, value=kv(2.0 ** 100), **shape), decay=0.5).check()
    b = Batch([64, 90], 4, 2, 64, 16, dtype, seed=8)
    b.scale = -0.3
    Run(b, decay=0.0).check()
    b.scale = 0.0
    Run(b, decay=-1.0).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("order", [1, -1])
def test_decode_value_scales_far_apart(dtype, order):
    """Value scales that rise (the unit moves again and again) or fall over the sequence, blocks of
    zeros among them."""
    rng = np.random.default_rng(9)
    n, block = 1600, 16
    size = 2.0 ** np.linspace(-12, 12, n // block)[::order].repeat(block)[:, None, None]
    value = size * rng.standard_normal((n, 2, 64))
    value[160:192], value[:16] = 0.0, 0.0
    Run(Batch([n], 6, 2, 64, block, dtype, seed=9, value=value), decay=1.0).check()
    value[:] = 0.0                                         # nothing but zeros
    r = Run(Batch([n], 6, 2, 64, block, dtype, seed=9, value=value), decay=1.0)
    r.check()
    assert not r.out.any()


@pytest.mark.parametrize("order", [1, -1])
def test_decode_rising_scores(order):
    # the running maximum moves at every tile, by more and more
    ramp = np.linspace(0.0, 60.0, 600)[::order, None, None] * np.ones((1, 1, 64))
    b = Batch([600], 4, 1, 64, 16, "bf16", seed=9, key=ramp)
    b.query = torch.ones_like(b.query)
    Run(b, decay=1.0).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("far,tokens,seqs", [(40, 100, 1), (3000, 5000, 1), (4999, 5000, 1), (70, 90, 400)])
def test_decode_scores_below_the_least_number_weigh_nothing(dtype, far, tokens, seqs):
    """The first `far` tokens' scores are beyond 32 bits, the others' are zero: the mean of
    the others' values, whose weights are equal.  Off are the products with the value scales and their
    rounding to fp16 (2^-11 + 2^-24; fp32 2^-22), sums (2^-23 an addition of 16 tokens) and the
    output's rounding."""
    key = np.zeros((tokens, 2, 64))
    key[:far] = 2000.0
    b = Batch([tokens], 4, 2, 64, 16, dtype, seed=far, key=key)
    b.query = rounded(np.full((1, 4, 64), -(2.0 ** 122)), dtype)
    ref, _, mass = b.reference()[:3]
    r = Run(b)
    r.tables, r.lens = r.tables.expand(seqs, -1).contiguous(), r.lens.expand(seqs).contiguous()
    r.query = r.query.expand(seqs, -1, -1).contiguous()
    r.out = torch.full_like(r.query, 77.0)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    weight = 2.0 ** -11 + 2.0 ** -24 if dtype == "bf16" else 2.0 ** -22
    bound = half * (1 + 2.0 ** -6) * np.abs(ref) + (weight + (tokens / 16 + 16) * 2.0 ** -23) * mass
    assert (np.abs(host(r()) - ref) <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [2.0 ** 14, 2.0 ** 24, 2.0 ** 27, 2.0 ** 34, 2.0 ** 60, 2.0 ** 110])
def test_decode_scores_with_steps_above_one(dtype, size):
    """Scores so large that neighbouring fp32 numbers are units or more apart: the token with
    the largest has all the weight (the next is further away than scores are off, twice), which is
    multiplied by its value scale and rounded once to fp16."""
    b = Batch([700, 33, 5000], 6, 2, 64, 16, dtype, seed=31, query_std=size)
    ref, _, _, _, reach = b.reference()
    sure = np.zeros(ref.shape[:2], dtype=bool)
    for r, n in enumerate(b.lens):
        at = np.arange(n)
        k, v = int8.read(b.cache, b.tables[r, at // 16].astype(np.int64) * 16 + at % 16)
        for h in range(6):
            x = np.sort(k[:, h // 3] @ host(b.query)[r, h]) * b.scale
            sure[r, h] = x[-1] - x[-2] > 2 * score_bound(reach[r, h, 0], 64) + 40
    assert sure.sum() >= 12
    got = host(Run(b)())
    half = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -21 if dtype == "bf16" else 2.0 ** -20
    assert np.isfinite(got).all()
    assert (np.abs(got - ref)[sure] <= half * np.abs(ref)[sure] + 1e-12).all()


def test_decode_nan_and_infinity():
    b = Batch([40, 60, 50], 4, 2, 64, 16, "bf16", seed=10)
    q = b.query.clone()
    q[0, 1, 5] = float("nan")
    q[2, 3, 9] = float("inf")
    b.query = q
    # a NaN key of sequence 1's first KV head, a NaN value of its second: their block's
    slot = b.slots[40 + 20]
    k, v = int8.read(b.cache, [slot])
    k[0, 0, 3], v[0, 1, 60] = np.nan, np.nan
    int8.write(b.cache, k, v, [slot])
    r = Run(b, decay=1.0)
    got = host(r())
    bad = np.zeros(got.shape, dtype=bool)
    bad[0, 1] = bad[2, 3] = bad[1] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    # the weights of all blocks that a NaN row attends
    w = host(r.new)
    assert np.isnan(w[0, :3]).all() and np.isnan(w[1, :4]).all() and np.isnan(w[2, :4]).all()


def test_decode_ignores_what_follows_a_sequence():
    """NaN scales and any codes in the blocks' later tiles' place cannot be: a block's scale is its
    tokens'.  But the tokens behind the last may hold anything."""
    b = Batch([5, 16, 130], 4, 2, 128, 64, "fp32", seed=35)
    first = Run(b, decay=1.0)
    first.check()
    for r, n in enumerate(b.lens):
        last = b.tables[r, (n - 1) // 64]
        raw = b.cache[last].view(np.uint8)
        for off in range((n - 1) % 64 + 1, 64):
            raw[:, off // 8, 16:].reshape(2, 2, 8, 8, 16)[:, :, :, off % 8] = 255 - 7 * off % 250
    again = Run(b, decay=1.0)
    assert torch.equal(again(), first.out) and torch.equal(again.new, first.new)


def test_decode_takes_strided_queries_and_padded_tables():
    b = Batch([5, 60, 33], 6, 2, 128, 16, seed=11, width=40)
    r = Run(b, decay=1.0)
    wide = torch.randn((3, 10 * 128), device="cuda").bfloat16()
    wide[:, 128:7 * 128] = r.query.flatten(1)
    r.query = wide[:, 128:7 * 128].unflatten(1, (6, 128))
    assert not r.query.is_contiguous()
    r.check()
    with pytest.raises(ValueError):
        pa.pa_decode_int8(r.out, r.query.transpose(0, 1).contiguous().transpose(0, 1), r.cache,
                          r.tables, r.lens, b.scale, r.ws)


def test_decode_length_errors_touch_nothing_else():
    b = Batch([16, 40, 8], 4, 2, 64, 16, seed=12, width=3)
    ref = b.reference()
    bound = decode_bound(ref[0], *ref[2:], b.lens, 64, "bf16")
    r = Run(b, decay=1.0)
    r.lens[0] = 49                       # three blocks hold 48
    got = r()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    assert (np.abs(host(got) - ref[0]) <= bound)[1:].all()
    assert (r.new[0] == 5).all() and (r.new[1] != 5).all() and (r.new[2, 0] != 5)
    r.lens[0] = -4                       # as an empty sequence
    r.lens[1] = (1 << 31) - 1
    r.new.fill_(5.0)
    got = r()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    assert not got[0].any() and (np.abs(host(got) - ref[0]) <= bound)[2].all()
    assert (r.new[:2] == 5).all()


@pytest.mark.parametrize("head,heads,tokens,bad", [(64, 4, 48, (1,)), (128, 8, 500, (60,)), (128, 8, 500, (61, 62)),
                                                   (256, 4, 500, tuple(range(40, 63))),
                                                   (64, 4, 500, tuple(range(0, 63, 3)))])
def test_decode_block_ids_outside_the_pool_count_as_zeros(head, heads, tokens, bad):
    shape = dict(heads=heads, kv_heads=1, head=head, block=8, seed=32)
    z = Batch([tokens], **shape)
    r = Run(Batch([tokens], **shape), decay=1.0)
    for i in bad:
        int8.write(z.cache, np.zeros((8, 1, head)), np.zeros((8, 1, head)),
                   z.tables[0, i].astype(np.int64) * 8 + np.arange(8))
    for off in (-1, z.cache.shape[0], -(1 << 31), (1 << 31) - 1):
        r.tables[0, list(bad)] = off
        ref = z.reference()
        assert_decode(r(), z, bad, ref)
        assert_weights(r.new, z, z.old, 1.0, np.full(z.old.shape, 5.0), bad, ref)
        assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID


def test_decode_weights_in_place_alone_and_none():
    b = Batch([30, 0, 70], 4, 2, 64, 16, seed=14)
    r = Run(b, decay=0.5)
    r.check()
    want = r.new.clone()
    mine = want != 5
    w = dev(b.old)
    args = (r.out, r.query, r.cache, r.tables, r.lens, b.scale, r.ws)
    pa.pa_decode_int8(*args, block_weights=w, decay=0.5)                  # in place
    assert torch.equal(w, torch.where(mine, want, dev(b.old)))
    w = torch.full_like(want, float("nan"))
    pa.pa_decode_int8(*args, block_weights_out=w, decay=0.5)              # from zeros
    assert torch.equal(torch.isnan(w), ~mine)
    _, ref, _, _, reach = b.reference()
    m = mine.cpu().numpy()
    assert (np.abs(host(w) - ref) <= weights_bound(ref, 0 * ref, reach, b.lens, 64))[m].all()
    before = r.cache.clone()
    big = torch.full((5, 4, 64), 33.0, dtype=torch.bfloat16, device="cuda")  # rows behind the batch stay
    pa.pa_decode_int8(big[:3], *args[1:])
    assert torch.equal(big[:3], r.out) and (big[3:] == 33).all() and torch.equal(before, r.cache)
    for bad in (dict(block_weights=w[:2]), dict(block_weights_out=w[:, :1]), dict(block_weights=w.T)):
        with pytest.raises(ValueError):
            pa.pa_decode_int8(*args, **bad)
    with pytest.raises(TypeError):
        pa.pa_decode_int8(*args, block_weights=w.double())


def test_decode_past_32_bit_offsets():
    # a pool of more than 4 GB; the sequence's blocks lie at its end
    blocks = 140_000
    cache = torch.zeros((blocks, 8, 2, 16 * 129), dtype=torch.int8, device="cuda")
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
    pa.pa_gather_cache_int8(ko, vo, cache, slots)
    rk, rv = held(b.cache, b.slots, "fp32")
    assert same(host(ko), rk) and same(host(vo), rv)
    pa.pa_reshape_and_cache_int8(cache, vo, ko, slots)
    want = b.cache.copy()
    int8.write(want, rv, rk, b.slots)
    assert_pool(cache[first:].cpu().numpy(), want, b.slots)
    assert not cache[:first].any()


def test_decode_many_sequences():
    lens = [1 + (i * 7) % 19 for i in range(3001)]
    Run(Batch(lens, 2, 1, 64, 8, seed=16), decay=1.0).check()


def test_decode_most_sequences():
    lens = [(i // 17) % 11 if i % 17 == 0 or i == 65534 else 0 for i in range(65535)]
    Run(Batch(lens, 2, 2, 64, 8, seed=24), decay=1.0).check()


@pytest.mark.parametrize("head,heads,hkv", [(64, 4, 2), (128, 2, 2), (256, 3, 3)])
@pytest.mark.parametrize("most,long", [(40, 0), (200, 0), (40, 9000), (300, 5000)])
def test_decode_short_sequences_beside_long_ones(head, heads, hkv, most, long):
    """Pairs that stay whole with a warp or a CTA, next to ones that are cut."""
    rng = np.random.default_rng(most + long + head)
    lens = rng.integers(0, most, 1500 if most < 100 else 300)
    lens[7::31] = 0
    if long:
        lens[[0, 150, len(lens) - 1]] = long, long - 3, long // 2
    Run(Batch(lens, heads, hkv, head, 16, seed=head + most), decay=1.0).check()


@pytest.mark.parametrize("head,heads,hkv", [(64, 8, 8), (128, 4, 4), (256, 5, 5)])
@pytest.mark.parametrize("longest", [510, 530, 1100])
def test_decode_pairs_about_as_long_as_may_stay_whole(head, heads, hkv, longest):
    rng = np.random.default_rng(longest + head)
    lens = rng.choice([1, 60, 480, 511, 512, 513, longest], 700, p=[.3, .3, .08, .08, .08, .08, .08])
    b = Batch([max(lens)], heads, hkv, head, 16, seed=head + longest)
    b.tables, b.lens = b.tables.repeat(len(lens), 0), lens.astype(np.int32)
    b.query = rounded(rng.standard_normal((len(lens), heads, head)), "bf16")
    b.old = rng.random(b.tables.shape).astype(np.float32)
    Run(b, decay=1.0).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_sequences_that_share_blocks_and_repeated_calls(dtype):
    """Rows of one table several times over, and calls that agree bit for bit
    however the parts of a sequence arrive."""
    b = Batch([5000, 77], 12, 2, 128, 16, dtype, seed=25)
    b.tables, b.lens = b.tables[[0, 1, 0, 0, 1]], b.lens[[0, 1, 0, 0, 1]]
    b.lens[3] = 4000
    b.old = b.old[[0, 1, 0, 0, 1]]
    b.query = rounded(np.random.default_rng(26).standard_normal((5, 12, 128)), dtype)
    r = Run(b, decay=1.0)
    r.check()
    first, weights = r.out.clone(), r.new.clone()
    for _ in range(20):
        assert torch.equal(r(), first) and torch.equal(r.new, weights)


@pytest.mark.parametrize("dtype,head,heads", [("bf16", 128, 4), ("bf16", 64, 16), ("bf16", 256, 8),
                                              ("fp32", 128, 4), ("fp32", 256, 8)])
def test_decode_sums_do_not_drift_with_the_length(dtype, head, heads):
    """Pairs of a million tokens, as many as warps and more, so that each sees about as much of one.
    Every value of an element is the same, so that the output is that value whatever the
    weights are.  Off are the weights' products with the value scale (2^-24) and roundings (bf16 2^-11,
    fp32 2^-22 at most), the output's (2^-8, 2^-24), the products at the end (2^-22) and two sums:
    chains of 2^12 tokens, steps of 16 or 32 that may cut off four times 2^-23, of which 2^7 at least and
    2^8 at most are added, rounded to nearest, 2^-24 / sqrt(3) in standard deviation each,
    of which ten are allowed (the sum of the weights: 2^9); then 2^8 chains' results likewise."""
    seqs, tokens, block = 2600, 1 << 20, 256
    value = np.resize([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -1.5], head) * (1 + np.arange(head) // 16 % 8)
    b = Batch([2048], heads, 1, head, block, dtype, seed=head + heads, query_std=2.0,
              value=np.broadcast_to(value, (2048, 1, head)))
    kept = int8.read(b.cache, b.slots[:1])[1][0]
    r = Run(b)
    r.tables = r.tables.repeat(1, tokens // 2048).expand(seqs, -1).contiguous()
    r.lens = torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")
    r.query = dev(rounded(2.0 * np.random.default_rng(head).standard_normal((seqs, heads, head)), dtype))
    r.out = torch.full_like(r.query, 77.0)
    worst = np.max(np.abs(host(r()) / kept - 1.0))
    deviation = 10 * 2.0 ** -24 / np.sqrt(3)
    weight, out = (2.0 ** -11, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -22, 2.0 ** -24)
    assert worst <= weight + out + 2.0 ** -22 + 2.0 ** -24 + 4 * 2.0 ** -23 + 2 * (2.0 ** 4.5 + 2.0 ** 4) * deviation
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,heads", [(64, 4), (64, 16), (128, 3), (128, 8), (128, 16), (256, 4), (256, 11)])
@pytest.mark.parametrize("rise", [0.0, 120.0, -120.0])
def test_decode_long_sequences_in_a_warp(dtype, head, heads, rise):
    """Pairs of several chains of 4096 tokens and a token, more than warps, whose scores
    stay, rise (the maximum moves again and again) or fall; value scales differ, so that the unit moves
    between chains too."""
    seqs, lens = 3000, [12289, 20001, 4096, 4097]
    rng = np.random.default_rng(head + heads)
    key = rng.standard_normal((20001, 1, head))
    key[:, 0, 0] = np.linspace(0.0, 6.0, 20001)
    b = Batch([20001], heads, 1, head, 64, dtype, seed=head + heads, key=key)
    q = host(b.query).repeat(4, 0)
    q[..., 0] = rise / (6.0 * b.scale)
    b.query, b.tables, b.lens = rounded(q, dtype), b.tables.repeat(4, 0), np.array(lens, dtype=np.int32)
    ref, weights, mass, total, reach = b.reference()
    bound = decode_bound(ref, mass, total, reach, b.lens, head, dtype)
    r = Run(b)
    r.tables, r.lens = r.tables.repeat(seqs // 4, 1), r.lens.repeat(seqs // 4)
    r.query = r.query.repeat(seqs // 4, 1, 1)
    r.out = torch.full_like(r.query, 77.0)
    r.decay, r.old, r.new = 1.0, None, torch.zeros(r.tables.shape, device="cuda")
    r.ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(r.cache, heads, r.tables), "cuda")
    got = host(r()).reshape((-1,) + ref.shape)
    assert (np.abs(got - ref) <= bound).all()
    got = host(r.new).reshape((-1,) + weights.shape)
    assert (np.abs(got - weights) <= weights_bound(weights, 0 * weights, reach, b.lens, head)).all()


def test_decode_fp32_keeps_small_weights():
    """One token far above all others, in warps that see whole sequences: the others'
    weights are 2^-34 to 2^-33 of its, and its value is zero.  Weights are kept in steps of
    2^-24 where the largest is 2^11 at least, so each is off by half a step, 2^-36 of the
    largest, at most, in units of up to twice the value scale (all values are 6 or zeros beside them);
    relative errors of what is kept are as in decode_bound."""
    seqs, tokens, heads, head = 2600, 8193, 8, 128
    key, value = np.full((tokens, 1, head), 0.0), np.full((tokens, 1, head), 6.0)
    key[..., 0], key[0, 0, 0], value[0] = -6.0, 6.0, 0.0
    b = Batch([tokens], heads, 1, head, 256, "fp32", seed=3, key=key, value=value)
    gap = np.linspace(33.0, 34.0, heads)                       # powers of two between the weights
    q = np.zeros((1, heads, head))
    q[0, :, 0] = gap * np.log(2.0) / (12.0 * b.scale)
    b.query = rounded(q, "fp32")
    ref, _, mass, total, reach = b.reference()
    r = Run(b)
    r.tables = r.tables.expand(seqs, -1).contiguous()
    r.lens = torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")
    r.query = r.query.expand(seqs, -1, -1).contiguous()
    r.out = torch.full_like(r.query, 77.0)
    bound = decode_bound(ref, mass, 0 * total, reach, [tokens], head, "fp32") + 2.0 ** -35 * total
    assert (np.abs(host(r()) - ref) <= bound).all()


def test_decode_takes_a_long_batch_over_shared_blocks():
    """4.3 billion tokens, as many sequences on one prefix have them (2^27 units of work and more)."""
    seqs, tokens, kinds = 65535, 65536, 16
    b = Batch([tokens], 4, 1, 128, 256, seed=29)
    b.query = rounded(np.random.default_rng(30).standard_normal((kinds, 4, 128)), "bf16")
    b.tables, b.lens = np.repeat(b.tables, kinds, 0), np.repeat(b.lens, kinds)
    ref, _, mass, total, reach = b.reference()
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
    # 65535 KV heads that hold one block, read 255 times by each of 130 sequences
    heads, seqs = 65535, 130
    cache = torch.zeros((1, heads, 16, 16 * 65), dtype=torch.int8, device="cuda")
    tables = torch.zeros((seqs + 1, 128), dtype=torch.int32, device="cuda")
    lens = torch.full((seqs + 1,), 128 * 128, dtype=torch.int32, device="cuda")
    lens[seqs] = 0
    q = torch.ones((seqs + 1, heads, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 77.0)
    ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(cache, heads), "cuda")
    pa.pa_decode_int8(out, q, cache, tables, lens, 1.0, ws)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    assert not out[seqs].any()
    lens[1:] = 0                                         # the same workspace, less work
    pa.pa_decode_int8(out, q, cache, tables, lens, 1.0, ws)
    assert pa.pa_get_device_error() == 0 and not out.any()


def test_refused_work_leaves_the_weights():
    heads, seqs = 4096, 2100
    cache = torch.zeros((1, heads, 16, 16 * 65), dtype=torch.int8, device="cuda")
    tables = torch.zeros((seqs, 64), dtype=torch.int32, device="cuda")
    lens = torch.full((seqs,), 64 * 128, dtype=torch.int32, device="cuda")
    q = torch.ones((seqs, heads, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.rand((seqs, 64), device="cuda")
    before, few = w.clone(), tables[:3]
    size = pa.pa_decode_int8_workspace_size(cache, heads, tables)
    assert size < 60e9
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    pa.pa_decode_int8(torch.empty_like(q), q, cache, tables, lens, 1.0, ws, block_weights=w)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    assert torch.equal(w, before)
    pa.pa_decode_int8(torch.empty_like(q[:3]), q[:3], cache, few, lens[:3], 1.0, ws, block_weights=w[:3])
    assert pa.pa_get_device_error() == 0
    # equal weights: a 64th of every head's attention for each block
    assert torch.allclose(w[:3], before[:3] + heads / 64, rtol=1e-4)


def test_two_graphs_share_a_workspace_and_lengths_grow():
    a = Run(Batch([70, 1, 300], 8, 2, 128, 16, seed=17), decay=0.5)
    b = Run(Batch([9, 2000], 4, 1, 128, 16, seed=18), decay=1.0)
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

    def check(r):
        ref = r.batch.reference()
        assert_decode(r.out, r.batch, reference=ref)
        assert_weights(r.new, r.batch, r.batch.old, r.decay, np.full(r.batch.old.shape, 5.0), reference=ref)

    for _ in range(3):
        a.out.fill_(5), b.out.fill_(5), a.new.fill_(5), b.new.fill_(5)
        for g in graphs:
            g.replay()
        check(a)
        check(b)
    # the captured call on shorter and on empty sequences
    for lens in ([33, 1, 299], [0, 0, 17], [0, 0, 0]):
        a.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        a.batch.lens = np.array(lens, dtype=np.int32)
        a.new.fill_(5)
        graphs[0].replay()
        check(a)


def test_two_streams_at_once():
    runs = [Run(Batch([900, 31, 40 + i], 8, 2, 64, 16, seed=19 + i), decay=1.0) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, s in zip(runs, streams):
            r(stream=s)
    torch.cuda.synchronize()
    for r in runs:
        ref = r.batch.reference()
        assert_decode(r.out, r.batch, reference=ref)
        assert_weights(r.new, r.batch, r.batch.old, 1.0, np.full(r.batch.old.shape, 5.0), reference=ref)


def test_decode_refuses_small_workspaces_and_buffers_in_them():
    r = Run(Batch([40], 4, 2, 64, 16))
    ws, r.ws = r.ws, r.ws[:-256]
    with pytest.raises(pa.PAError) as e:
        r()
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    r.ws, r.decay = ws, 1.0              # large enough without weights, too small with them
    with pytest.raises(pa.PAError):
        r()
    need = pa.pa_decode_int8_workspace_size(r.cache, 4, r.tables)
    assert need > ws.numel()
    arena = torch.zeros(need + 8192, dtype=torch.uint8, device="cuda")
    r.ws = arena[:need]
    at = (need + 15) // 16 * 16
    for name in ("out", "query", "cache", "tables", "lens", "new", "old"):
        was = getattr(r, name)
        inside = arena[at - 16:at - 16 + was.nbytes] if name != "cache" else arena[:was.nbytes]
        setattr(r, name, inside.view(was.dtype).view(was.shape))
        with pytest.raises(pa.PAError) as e:
            r()
        assert e.value.status == pa.PA_ERR_INVALID_ARG, name
        setattr(r, name, was)
    r.out = arena[at:at + r.out.nbytes].view(r.out.dtype).view(r.out.shape)
    r.check()


def test_decode_waits_that_give_up_leave_the_workspace_usable():
    # A limit of one cycle, and more to read than L2 holds, so that most waits
    # for a copy find it not yet there and give up.
    head, hkv, block, lens = 128, 8, 16, [120_000, 5, 0, 60_001]
    counts = [-(-n // block) for n in lens]
    cache = torch.randint(-128, 128, (sum(counts), hkv, block // 8, 16 * (head + 1)), dtype=torch.int8,
                          device="cuda")
    cache.view(torch.uint8)[..., :8] = torch.tensor([0.01, 0.02], device="cuda").view(torch.uint8)
    tables = torch.zeros((4, max(counts)), dtype=torch.int32)
    ids, at = torch.randperm(sum(counts)).int(), 0
    for r, c in enumerate(counts):
        tables[r, :c] = ids[at:at + c]
        at += c
    tables, lens = tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((4, 16, head), device="cuda").bfloat16()
    ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(cache, 16), "cuda")

    def call():
        out = torch.full_like(q, 5.0)
        pa.pa_decode_int8(out, q, cache, tables, lens, head ** -0.5, ws)
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


@pytest.mark.parametrize("heads,in_place", [(16, True), (16, False), (8, True)])
def test_waits_that_give_up_leave_the_weights(heads, in_place):
    """The sums of the blocks' weights need every cell and row of the call: where a wait gave up
    the weights stay, as they last over steps; the next call's are right again."""
    head, hkv, block, lens = 128, 8, 16, [120_000, 5, 0, 60_001]
    counts = [-(-n // block) for n in lens]
    cache = torch.randint(-128, 128, (sum(counts), hkv, block // 8, 16 * (head + 1)), dtype=torch.int8,
                          device="cuda")
    cache.view(torch.uint8)[..., :8] = torch.tensor([0.01, 0.02], device="cuda").view(torch.uint8)
    tables = torch.zeros((4, max(counts)), dtype=torch.int32)
    ids, at = torch.randperm(sum(counts)).int(), 0
    for r, c in enumerate(counts):
        tables[r, :c] = ids[at:at + c]
        at += c
    tables, lens = tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((4, heads, head), device="cuda").bfloat16()
    ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(cache, heads, tables), "cuda")
    before = torch.rand(tables.shape, device="cuda")

    def call(weights=True):
        w, new = before.clone(), None if in_place else torch.full_like(before, 7.0)
        kw = dict(block_weights=w, block_weights_out=new, decay=0.5) if weights else {}
        out = torch.empty_like(q)
        pa.pa_decode_int8(out, q, cache, tables, lens, head ** -0.5, ws, **kw)
        assert in_place or torch.equal(w, before)
        return out, w if in_place else new

    out, first = call()
    assert pa.pa_get_device_error() == 0 and torch.isfinite(first).all()
    mine = torch.arange(tables.shape[1], device="cuda") < torch.tensor(counts, device="cuda")[:, None]
    added = (first - 0.5 * before)[mine].double().sum()
    assert abs(added - 3 * heads) < 1e-3 * heads              # each row's attention once
    kept = before if in_place else torch.full_like(before, 7.0)
    for calls in ((True,), (True, True), (False,), (False, True)):   # with weights or without
        pa.pa_set_decode_wait_limit(1)
        try:
            for weights in calls:
                assert torch.equal(call(weights)[1], kept)
                assert pa.pa_get_device_error() == pa.PA_DEVERR_TIMEOUT
        finally:
            pa.pa_set_decode_wait_limit(0)
        for _ in range(2):
            got = call()
            assert torch.equal(got[0], out) and torch.equal(got[1], first)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("width,seqs", [(40, 3), (5000, 70), (8192, 300)])
def test_weights_over_tables_wider_than_the_sequences(width, seqs):
    lens = np.random.default_rng(width).integers(0, 300, seqs)
    lens[:3] = [0, 16 * min(width, 40), 1]
    r = Run(Batch(lens, 4, 2, 64, 16, seed=width, width=width), decay=0.5)
    r.check()
    r.lens[2] = 16 * width + 1                                # past its row: its weights stay
    r.batch.lens[2] = 0
    r.new.fill_(5.0)
    ref = r.batch.reference()
    r()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_SEQ_LEN
    assert_weights(r.new, r.batch, r.batch.old, 0.5, np.full(r.batch.old.shape, 5.0), reference=ref)


def test_weights_cost_what_the_sequences_have_not_what_the_tables_could():
    """256 sequences of seven blocks in tables of 8192 columns: at most three times as long as in tables
    that just hold them (a length per entry is looked at; reading every entry's cells takes 14 times as
    long)."""
    seqs, tokens, heads, hkv, head = 256, 100, 32, 8, 128
    n = -(-tokens // 16)
    cache = pa.alloc_int8_cache(seqs * n, 16, hkv, head)
    q = torch.randn((seqs, heads, head), device="cuda").bfloat16()
    out, lens = torch.empty_like(q), torch.full((seqs,), tokens, dtype=torch.int32, device="cuda")

    def us(width):
        t = torch.zeros((seqs, width), dtype=torch.int32, device="cuda")
        t[:, :n] = torch.arange(seqs * n, device="cuda").int().view(seqs, n)
        w = torch.zeros(t.shape, device="cuda")
        ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(cache, heads, t), "cuda")
        call = lambda: pa.pa_decode_int8(out, q, cache, t, lens, head ** -0.5, ws, block_weights=w)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                call()
        best = float("inf")
        for _ in range(8):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert us(8192) < 3 * us(n)
