"""Pins of the 4-bit pool's oracle against other sources (torch's e4m3,
fixed numbers, closed forms, the binary64 decode of the 16-bit oracle), and
the refusals of the library's entry points, which need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_78_gb300 as pa

from fp4_util import Batch, host
from oracle import fp4


def test_e4m3_table_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), fp4.E4M3)
    x = np.random.default_rng(0).uniform(0, 460, 20000) ** 2 / 460
    x = np.concatenate([x, fp4.E4M3, (fp4.E4M3[1:] + fp4.E4M3[:-1]) / 2])  # ties among them
    x = np.minimum(x, 448.0).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp4.nearest_code(fp4.E4M3, x.astype(np.float64)), want)


def test_e2m1_borders_go_to_even_codes():
    # 0 0.5 1 1.5 2 3 4 6: halfway points and the code with an even index
    borders = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for b, code in borders.items():
        assert fp4.nearest_code(fp4.E2M1, np.array([b]))[0] == code
        below = fp4.nearest_code(fp4.E2M1, np.array([b * (1 - 2 ** -20)]))[0]
        above = fp4.nearest_code(fp4.E2M1, np.array([b * (1 + 2 ** -20)]))[0]
        assert above == below + 1 and code in (below, above)
    assert fp4.nearest_code(fp4.E2M1, np.array([1e9]))[0] == 7


def test_rounding_error_is_bounded_and_idempotent():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 3, 128)) * np.exp(rng.standard_normal((50, 3, 1)))
    codes, scales = fp4.quantise(x, 0.5)
    y = fp4.dequantise(codes, scales, 0.5)
    top = np.abs(x.reshape(50, 3, 8, 16)).max(-1, keepdims=True)
    # half of the widest gap (1 scale) or the cut at 6: the scale is at most
    # 2^-4 above and below max / 6
    err = np.abs(x - y).reshape(50, 3, 8, 16)
    assert (err <= top / 6 * (1 + 2 ** -4) * (1 + 1e-9)).all()
    assert np.array_equal(fp4.dequantise(*fp4.quantise(y, 0.5), 0.5), y)


def test_special_values():
    x = np.zeros((4, 16))
    x[0, 3] = np.nan
    x[1, 5] = -np.inf
    x[2, :] = 1e-30
    codes, scales = fp4.quantise(x)
    y = fp4.dequantise(codes, scales)
    assert np.isnan(y[0]).all()
    assert y[1, 5] == -6 * 448 and (y[1, :5] == 0).all()
    assert (y[2] == 0).all() and (y[3] == 0).all()


@pytest.mark.parametrize("head,block", [(64, 8), (128, 16), (256, 32)])
def test_write_and_read_round_trip_and_touch_only_their_rows(head, block):
    rng = np.random.default_rng(head)
    cache = rng.integers(0, 256, (5, 2, block // 8, 9 * head), dtype=np.uint8)
    slots = rng.permutation(5 * block)[:11].astype(np.int64)
    slots[4] = -1
    k, v = rng.standard_normal((2, 11, 2, head))
    others = np.setdiff1d(np.arange(5 * block), slots)
    before = fp4.read(cache, others)
    fp4.write(cache, k, v, slots, 2.0, 0.5)
    for a, b in zip(before, fp4.read(cache, others)):
        assert np.array_equal(a, b, equal_nan=True)
    live = slots >= 0
    gk, gv = fp4.read(cache, slots[live], 2.0, 0.5)
    assert np.array_equal(gk, fp4.dequantise(*fp4.quantise(k, 2.0), 2.0)[live])
    assert np.array_equal(gv, fp4.dequantise(*fp4.quantise(v, 0.5), 0.5)[live])


def test_tile_layout_on_a_marked_row():
    # token 3 of the second tile of block 1: one key element, one value element
    cache = np.zeros((2, 1, 2, 9 * 64), dtype=np.uint8)
    k, v = np.zeros((2, 1, 1, 64))
    k[0, 0, 37] = 6.0   # group 2, byte 18 of the row, high nibble
    v[0, 0, 20] = -6.0  # group 1, byte 2 of the group, low nibble
    fp4.write(cache, k, v, [16 + 8 + 3])
    tile = cache[1, 0, 1]
    want = np.zeros(9 * 64, dtype=np.uint8)
    want[3 * 32 + 18] = 7 << 4
    want[4 * 64 + 1 * 64 + 3 * 8 + 2] = 15
    want[8 * 64 + 3 * 4 + 2] = 0x38        # e4m3 of 1
    want[8 * 64 + 32 + 1 * 8 + 3] = 0x38
    assert np.array_equal(tile, want) and not cache[0].any() and not cache[1, 0, 0].any()


def test_decode_agrees_with_the_16_bit_oracle():
    b = Batch([0, 1, 9, 70], 6, 2, 64, 16, "fp32", seed=3)
    ref, mass, total, reach = b.reference()
    k, v = fp4.read(b.cache, np.arange(b.cache.shape[0] * 16))
    cache = np.stack([k, v]).reshape(2, -1, 16, 2, 64).astype(np.float32)  # exact
    got = oracle.decode(host(b.query).astype(np.float32), np.nan_to_num(cache), b.tables, b.lens,
                        b.scale)
    assert np.abs(got - ref).max() < 1e-12
    assert (np.abs(ref) <= mass + 1e-12).all() and (mass <= total + 1e-12).all()
    assert (reach[1:] > 0).all()


def test_extend_tables_agrees_with_the_host_pool():
    pool = pa.Pool(40, 8)
    prompts = [5, 8, 0, 17]
    seqs = [pool.add_seq(n) for n in prompts]
    tables, lens = pool.fill_tables(seqs, 6)
    ring = pool.free_queue()
    state = [0, len(ring)]
    t, length = tables.numpy(), lens.numpy()
    for _ in range(9):  # nine decode steps
        slots, _ = pool.append_tokens(seqs)
        t, length, state, got, pos, starts, refused = fp4.extend_tables(
            t, length, [1, 1, 1, 1], 8, 40, 4, ring, state)
        assert not refused and np.array_equal(got, slots.numpy())
        want, want_lens = pool.fill_tables(seqs, 6)
        used = np.arange(6) < -(-want_lens.numpy()[:, None] // 8)
        assert np.array_equal(np.where(used, t, 0), want.numpy())
        assert np.array_equal(length, want_lens.numpy())
    assert state[1] == pool.num_free()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

P = ctypes.c_void_p(256)


def far(i):
    """A buffer's address, away from the others'."""
    return ctypes.c_void_p(i << 24)


def desc(**kw):
    d = dict(num_blocks=16, block_size=16, num_kv_heads=2, head_size=64, dtype=pa.PA_FP4)
    d.update(kw)
    return pa.CacheDesc(**d)


def write_call(d=None, **kw):
    d = desc() if d is None else d
    return pa.lib.pa_reshape_and_cache_fp4(
        kw.get("cache", far(1)), ctypes.byref(d), kw.get("key", far(2)), kw.get("value", far(3)),
        kw.get("dtype", pa.PA_BF16), kw.get("ks", 128), kw.get("vs", 128), kw.get("slots", P),
        kw.get("n", 4), kw.get("key_scale", 1.0), kw.get("value_scale", 1.0), None)


def gather_call(d=None, **kw):
    d = desc() if d is None else d
    return pa.lib.pa_gather_cache_fp4(
        kw.get("key", far(2)), kw.get("value", far(3)), kw.get("dtype", pa.PA_BF16),
        kw.get("cache", far(1)),
        ctypes.byref(d), kw.get("slots", P), kw.get("n", 4), kw.get("key_scale", 1.0),
        kw.get("value_scale", 1.0), None)


def decode_call(d=None, **kw):
    d = desc() if d is None else d
    return pa.lib.pa_decode_fp4(
        kw.get("out", far(2)), kw.get("query", far(3)), kw.get("dtype", pa.PA_BF16),
        kw.get("qs", 14 * 64), kw.get("cache", far(1)), ctypes.byref(d), kw.get("key_scale", 1.0), kw.get("value_scale", 1.0),
        P, kw.get("mb", 4), P, kw.get("s", 2), kw.get("heads", 14), kw.get("scale", 0.125),
        kw.get("ws", P), kw.get("ws_bytes", 1 << 30), None)


@pytest.mark.parametrize("call", [write_call, gather_call, decode_call])
@pytest.mark.parametrize("bad", [dict(dtype=pa.PA_BF16), dict(block_size=4), dict(block_size=24),
                                 dict(block_size=512), dict(num_blocks=0), dict(num_kv_heads=0),
                                 dict(head_size=0)])
def test_bad_pools_are_refused(call, bad):
    assert call(desc(**bad)) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [write_call, gather_call, decode_call])
def test_bad_arguments_are_refused(call):
    assert call(desc(head_size=96)) == pa.PA_ERR_UNSUPPORTED
    assert call(dtype=pa.PA_FP4) == pa.PA_ERR_INVALID_ARG
    assert call(dtype=7) == pa.PA_ERR_INVALID_ARG
    for bad in (0.0, -1.0, 3.0, 0.1, float("nan"), float("inf"), 2.0 ** 33, 2.0 ** -33):
        assert call(key_scale=bad) == pa.PA_ERR_INVALID_ARG
        assert call(value_scale=bad) == pa.PA_ERR_INVALID_ARG
    assert call(cache=None) == pa.PA_ERR_INVALID_ARG
    assert call(cache=ctypes.c_void_p(264)) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [write_call, gather_call])
def test_bad_rows_are_refused(call):
    assert call(n=-1) == pa.PA_ERR_INVALID_ARG
    assert call(n=0, cache=None, key=None, value=None, slots=None) == pa.PA_OK
    for name in ("key", "value"):
        assert call(**{name: None}) == pa.PA_ERR_INVALID_ARG
        assert call(**{name: ctypes.c_void_p(264)}) == pa.PA_ERR_INVALID_ARG
    assert call(slots=None) == pa.PA_ERR_INVALID_ARG
    assert call(slots=ctypes.c_void_p(260)) == pa.PA_ERR_INVALID_ARG


def test_bad_strides_are_refused():
    for name in ("ks", "vs"):
        for bad in (0, -128, 120, 132):  # 132 bf16 elements: not a multiple of 16 bytes
            assert write_call(**{name: bad}) == pa.PA_ERR_INVALID_ARG
    assert write_call(dtype=pa.PA_FP32, ks=130) == pa.PA_ERR_INVALID_ARG


def test_decode_refusals():
    assert decode_call(heads=13) == pa.PA_ERR_INVALID_ARG
    assert decode_call(heads=0) == pa.PA_ERR_INVALID_ARG
    assert decode_call(heads=34) == pa.PA_ERR_UNSUPPORTED      # a group of 17
    assert decode_call(s=-1) == pa.PA_ERR_INVALID_ARG
    assert decode_call(s=65536) == pa.PA_ERR_INVALID_ARG
    assert decode_call(s=0, out=None, ws=None) == pa.PA_OK
    assert decode_call(mb=0) == pa.PA_ERR_INVALID_ARG
    for bad in (float("nan"), float("inf")):
        assert decode_call(scale=bad) == pa.PA_ERR_INVALID_ARG
    assert decode_call(qs=13 * 64) == pa.PA_ERR_INVALID_ARG
    assert decode_call(qs=14 * 64 + 4) == pa.PA_ERR_INVALID_ARG
    for name in ("out", "query", "ws"):
        assert decode_call(**{name: None}) == pa.PA_ERR_INVALID_ARG
        assert decode_call(**{name: ctypes.c_void_p(264)}) == pa.PA_ERR_INVALID_ARG


def test_16_bit_calls_refuse_a_4_bit_pool():
    d = desc()
    assert pa.lib.pa_reshape_and_cache(P, ctypes.byref(d), P, P, P, 4, None) == pa.PA_ERR_INVALID_ARG
    assert pa.lib.pa_decode(P, P, P, ctypes.byref(d), P, 4, P, 2, 14, 0.125, 64, 0, P, 1 << 20,
                            None) == pa.PA_ERR_INVALID_ARG
    b = desc(dtype=pa.PA_BF16)
    assert pa.lib.pa_swap_blocks(P, ctypes.byref(d), P, ctypes.byref(b), P, 1,
                                 None) == pa.PA_ERR_INVALID_ARG
    assert pa.lib.pa_copy_blocks(P, ctypes.byref(desc(block_size=4)), P, 1,
                                 None) == pa.PA_ERR_INVALID_ARG


def tables_call(**kw):
    g = kw.get
    return pa.lib.pa_extend_tables(
        g("tables", far(1)), g("mb", 4), g("lens", far(2)), g("new", far(3)), g("n", 2),
        g("bs", 16), g("nb", 9), g("ring", far(4)), g("cap", 5), g("state", far(5)),
        g("lens_out", far(6)), g("state_out", far(7)), g("slots", far(8)), g("pos", far(9)),
        g("starts", far(10)), g("most", 8), None)


def test_table_refusals():
    bad = [dict(n=-1), dict(n=8193), dict(mb=0), dict(bs=12), dict(bs=512), dict(nb=0),
           dict(most=-1), dict(most=(1 << 30) + 1), dict(most=1 << 26), dict(tables=None), dict(lens=None),
           dict(new=None), dict(lens_out=None), dict(slots=None), dict(ring=None),
           dict(state=None), dict(state_out=None), dict(cap=0), dict(cap=-3),
           dict(cap=(1 << 30) + 1), dict(slots=ctypes.c_void_p(260)),
           dict(pos=ctypes.c_void_p(258)), dict(starts=ctypes.c_void_p(257)),
           dict(ring=None, state=None, state_out=None)]  # a capacity without a ring
    for kw in bad:
        assert tables_call(**kw) == pa.PA_ERR_INVALID_ARG, kw


def test_overlapping_buffers_are_refused():
    # two requests: 8 bytes of lengths, counts and state, 12 of starts, 20 of the
    # ring, 32 of the tables and of positions, 64 of slots
    sizes = dict(tables=32, lens=8, new=8, ring=20, state=8, lens_out=8, state_out=8, slots=64,
                 pos=32, starts=12)
    where = dict(tables=1, lens=2, new=3, ring=4, state=5, lens_out=6, state_out=7, slots=8, pos=9,
                 starts=10)
    written = ("tables", "lens_out", "state_out", "slots", "pos", "starts")
    for a in written:
        for b in sizes:
            if b == a:
                continue
            step = 8 if a == "slots" else 4
            at = where[b] << 24
            # a's last element on b's first, and a's first on b's last
            first = at - sizes[a] + step
            last = at + (sizes[b] - 4) // step * step
            for x in (first, last):
                assert tables_call(**{a: ctypes.c_void_p(x)}) == pa.PA_ERR_INVALID_ARG, (a, b)
    assert tables_call(lens_out=far(3)) == pa.PA_ERR_INVALID_ARG   # in place of the counts
    assert tables_call(state_out=far(2)) == pa.PA_ERR_INVALID_ARG
    # four rows of 256 bytes; a pool of 16 blocks
    row, pool = 4 * 256, 16 * 2 * 2 * 9 * 64
    for x in (16, row - 16):
        assert gather_call(key=ctypes.c_void_p((3 << 24) + x)) == pa.PA_ERR_INVALID_ARG
        assert gather_call(key=ctypes.c_void_p((3 << 24) - x)) == pa.PA_ERR_INVALID_ARG
    for name in ("key", "value"):
        assert gather_call(**{name: ctypes.c_void_p((1 << 24) - row + 16)}) == pa.PA_ERR_INVALID_ARG
        assert gather_call(**{name: ctypes.c_void_p((1 << 24) + pool - 16)}) == pa.PA_ERR_INVALID_ARG
    # two rows of 14 heads, and rows 2000 elements apart
    assert decode_call(out=far(3)) == pa.PA_ERR_INVALID_ARG
    assert decode_call(out=ctypes.c_void_p((3 << 24) + 2 * 2 * 896 - 16)) == pa.PA_ERR_INVALID_ARG
    assert decode_call(out=ctypes.c_void_p((3 << 24) - 2 * 2 * 896 + 16)) == pa.PA_ERR_INVALID_ARG
    assert decode_call(qs=2000, out=ctypes.c_void_p((3 << 24) + 2 * 2896 - 16)) == pa.PA_ERR_INVALID_ARG


def test_writes_that_overlap_what_is_read_are_refused():
    """First and last elements of one buffer on the last and first of another."""
    row, pool, slots = 4 * 256, 16 * 2 * 2 * 9 * 64, 4 * 8
    at = ctypes.c_void_p
    for name, size, step in (("key", row, 16), ("value", row, 16), ("slots", slots, 8)):
        for x in ((1 << 24) - size + step, 1 << 24, (1 << 24) + pool - 16):
            assert write_call(**{name: at(x)}) == pa.PA_ERR_INVALID_ARG, name
    # rows 2000 elements apart reach into the cache with their last one
    assert write_call(ks=2000, key=at((1 << 24) - 2 * (3 * 2000 + 128) + 16)) == pa.PA_ERR_INVALID_ARG
    for out in (2, 3):
        for x in ((out << 24) - slots + 8, out << 24, (out << 24) + row - 8):
            assert gather_call(slots=at(x)) == pa.PA_ERR_INVALID_ARG
    # two rows of 14 heads of 64, tables of two rows of four, two lengths
    def decode(**kw):
        g = lambda name, i: kw.get(name, far(i))
        return pa.lib.pa_decode_fp4(g("out", 2), g("query", 3), pa.PA_BF16, 14 * 64, g("cache", 1),
                                    ctypes.byref(desc()), 1.0, 1.0, g("tables", 4), 4, g("lens", 5), 2,
                                    14, 0.125, g("ws", 64), 1 << 30, None)
    size = 2 * 14 * 64 * 2
    for name, i, other, step in (("cache", 1, pool, 16), ("tables", 4, 32, 4), ("lens", 5, 8, 4)):
        for x in ((2 << 24) - other + step, 2 << 24, (2 << 24) + size - step):
            if name != "cache" or x % 16 == 0:
                assert decode(**{name: at(x)}) == pa.PA_ERR_INVALID_ARG, name
        for x in ((i << 24) - size + 16, (i << 24) + (other - 4) // 16 * 16):
            assert decode(out=at(x)) == pa.PA_ERR_INVALID_ARG, name


def test_python_refusals():
    c = torch.zeros((4, 2, 2, 9 * 64), dtype=torch.uint8)
    d = pa.fp4_cache_desc(c)
    assert (d.num_blocks, d.block_size, d.num_kv_heads, d.head_size) == (4, 16, 2, 64)
    with pytest.raises(TypeError):
        pa.fp4_cache_desc(c.float())
    with pytest.raises(ValueError):
        pa.fp4_cache_desc(c[..., :100])
    with pytest.raises(ValueError):
        pa.fp4_cache_desc(c[:, :, :, ::3][..., :9])
    with pytest.raises(ValueError):
        pa.alloc_fp4_cache(4, 4, 2, 64, device="cpu")
    assert pa.alloc_fp4_cache(4, 16, 2, 64, device="cpu").shape == c.shape
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):                      # host tensors
        pa.pa_reshape_and_cache_fp4(c, k, k, s)
    with pytest.raises(TypeError):
        pa.pa_reshape_and_cache_fp4(c, k, k.float(), s)
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache_fp4(c, k, k[:2], s)
    with pytest.raises(ValueError):
        pa.pa_gather_cache_fp4(k[:, :1], k[:, :1], c, s)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_decode_fp4(q, q, c, t[:1], n, 1.0, s)
    with pytest.raises(TypeError):
        pa.pa_decode_fp4(q.float(), q, c, t, n, 1.0, s)
    with pytest.raises(ValueError):
        pa.pa_extend_tables(t, n, n, 16, 4, s, token_starts=n)
    with pytest.raises(ValueError):
        pa.pa_extend_tables(t, n, n, 16, 4, s, free_blocks=n)
    with pytest.raises(ValueError):
        pa.pa_extend_tables(t, n, n, 16, 4, s)           # host tensors


def test_sizes_past_32_bits_are_refused():
    """Not cut to 32 bits, where they could pass for small ones."""
    meta = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="meta")
    big = (1 << 32) + 8
    lens, slots = meta(1), meta(8, dtype=torch.int64)
    for kw in (dict(tables=meta(1, big)), dict(slots=meta(big, dtype=torch.int64)), dict(blocks=big),
               dict(size=big), dict(ring=meta(big))):
        ring = kw.get("ring")
        with pytest.raises(ValueError, match="past 2"):
            pa.pa_extend_tables(kw.get("tables", meta(1, 4)), lens, lens, kw.get("size", 16),
                                kw.get("blocks", 9), kw.get("slots", slots), free_blocks=ring,
                                free_state=None if ring is None else meta(2))
    q = meta(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="past 2"):
        pa.pa_decode_fp4(q, q, meta(4, 2, 2, 9 * 64, dtype=torch.uint8), meta(1, big), lens, 1.0, slots)


@pytest.mark.parametrize("block", [-16, 0, 7, 12, 24, 512])
def test_pools_that_no_call_takes_are_not_allocated(block):
    with pytest.raises(ValueError):
        pa.alloc_fp4_cache(4, block, 2, 64, device="cpu")


def test_workspace_size_refusals():
    out = ctypes.c_size_t()
    call = lambda d, h: pa.lib.pa_decode_fp4_workspace_size(ctypes.byref(d), h, ctypes.byref(out))
    assert call(desc(dtype=pa.PA_BF16), 4) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 3) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 0) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 34) == pa.PA_ERR_UNSUPPORTED
    assert call(desc(head_size=32), 4) == pa.PA_ERR_UNSUPPORTED
