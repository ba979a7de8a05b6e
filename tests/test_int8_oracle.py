"""The 8-bit pool's, the eviction's and the norms' oracle against definitions of its own,
and the calls' refusals (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_78_gb300 as pa
from int8_util import Batch, host, rounded
from oracle import int8


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def empty(blocks, heads, block, head, seed=None):
    if seed is None:
        return np.zeros((blocks, heads, block // 8, 16 * (head + 1)), dtype=np.int8)
    return np.random.default_rng(seed).integers(-128, 128, (blocks, heads, block // 8, 16 * (head + 1)),
                                                dtype=np.int8)


def test_tile_layout_on_a_marked_token():
    cache = empty(3, 2, 16, 64)
    key = np.zeros((2, 2, 64))
    value = np.zeros((2, 2, 64))
    key[1, 1, 37], value[1, 1, 5] = 127.0, -254.0
    int8.write(cache, key, value, [16, 27])          # block 1, offsets 0 and 11
    raw = cache.view(np.uint8)
    for tile in range(2):                            # scales are repeated in every tile
        assert raw[1, 1, tile, :8].view(np.float32).tolist() == [1.0, 2.0]
        assert not raw[1, 1, tile, 8:16].any() and not raw[1, 0, tile, :16].any()
    tile = raw[1, 1, 1]
    assert tile[16 + 37 // 16 * 128 + 3 * 16 + 37 % 16] == 255
    assert tile[16 + 8 * 64 + 3 * 16 + 5] == 1
    assert (tile[16:] == 128).sum() + (tile[16:] == 0).sum() == 16 * 64 - 2
    k, v = int8.read(cache, [27])
    assert k[0, 1, 37] == 127 and v[0, 1, 5] == -254 and np.abs(k).sum() == 127 and np.abs(v).sum() == 254
    assert not raw[[0, 2]].any()


@pytest.mark.parametrize("head,block", [(64, 8), (128, 16), (256, 32)])
def test_rounding_error_is_half_a_step_of_the_block(head, block):
    rng = np.random.default_rng(head)
    cache = empty(4, 2, block, head, seed=1)
    n = 2 * block + 3
    slots = np.concatenate([3 * block + np.arange(block), block + np.arange(block), np.arange(3)])
    key, value = rng.standard_normal((n, 2, head)), 0.01 * rng.standard_normal((n, 2, head))
    int8.write(cache, key, value, slots)
    for got, x in zip(int8.read(cache, slots), (key, value)):
        for b in np.unique(slots // block):
            at = slots // block == b
            step = np.abs(x[at]).max((0, 2)) / 127
            assert (np.abs(got[at] - x[at]).max((0, 2)) <= step * (0.5 + 2.0 ** -17)).all()


def test_scales_grow_and_blocks_begin_anew():
    cache = empty(2, 1, 8, 64, seed=2)
    x = np.zeros((1, 1, 64))

    def put(v, off):
        x[0, 0, 0] = v
        int8.write(cache, x, x, [8 + off])
        return float(int8.block_scales(cache, 1, 0)[0, 0])

    assert put(127.0, 0) == 1.0                       # begins
    assert put(3.0, 1) == 1.0                         # fits
    assert put(254.0, 2) == 2.0                       # grows: 3 becomes 2 * rint(1.5), a tie to 2
    assert int8.read(cache, [8, 9, 10])[0][:, 0, 0].tolist() == [128.0, 4.0, 254.0]
    assert np.isnan(put(np.inf, 3)) and np.isnan(put(1.0, 4))
    assert np.isnan(int8.read(cache, [8])[0]).all()
    assert put(12.7, 0) == np.float32(12.7 / 127)     # begins anew
    both = np.ones((2, 1, 64))
    int8.write(cache, both, both, [12, 8])            # one of the call's tokens is the first
    assert float(int8.block_scales(cache, 1, 1)[0, 0]) == np.float32(1 / 127)


def test_decode_agrees_with_the_16_bit_oracle():
    b = Batch([0, 1, 9, 70], 6, 2, 64, 16, "fp32", seed=3)
    ref, weights, mass, total, reach = b.reference()
    k, v = int8.read(b.cache, np.arange(b.cache.shape[0] * 16))
    cache = np.stack([k, v]).reshape(2, -1, 16, 2, 64)
    # 64 bits of code * scale rounded to 32: the outputs move by about 2^-24 of the values
    got = oracle.decode(host(b.query).astype(np.float32), np.nan_to_num(cache, posinf=0, neginf=0).astype(np.float32),
                        b.tables, b.lens, b.scale)
    assert (np.abs(got - ref) <= 2.0 ** -20 * (mass + 1e-9)).all()
    assert (np.abs(ref) <= mass + 1e-12).all() and (mass <= total + 1e-9).all()
    assert (reach[1:] > 0).all()
    assert np.allclose(weights.sum(1), [0, 6, 6, 6])
    one = np.zeros(5)
    one[0] = 6
    assert np.allclose(weights[1], one)


def test_eviction_by_hand():
    nan = np.nan
    tables = np.array([[10, 11, 12, 13, 14, -1], [20, 21, 22, -1, -1, -1], [30, 31, 32, 33, 34, 35]])
    weights = np.array([[1, 5, 2, 2, 9, 7], [3, 1, 2, 7, 7, 7], [nan, 0.0, nan, -0.0, -4, 1]], dtype=np.float32)
    t, w, n, ring, state, gone, refused = int8.evict(tables, weights, [79, 33, 96], 16, 3, 1, 1,
                                                     [90, 91, 92, 93, 94, 95, 96, 97], [6, 3], [0, 16, 0])
    # row 0 gives up blocks 2 and 3 (both 2, among 1 .. 3), row 1 nothing, row 2 blocks 4, 1, 3
    assert t.tolist() == [[10, 11, 14, 12, 13, -1], [20, 21, 22, -1, -1, -1], [30, 32, 35, 31, 33, 34]]
    assert np.array_equal(w, np.array([[1, 5, 9, 0, 0, 7], [3, 1, 2, 7, 7, 7], [nan, nan, 1, 0, 0, 0]]), equal_nan=True)
    assert n.tolist() == [47, 33, 48] and gone.tolist() == [32, 16, 48] and not refused
    assert state == [6, 8] and ring.tolist() == [92 - 2, 12, 13, 31, 33, 34, 96, 97]
    for bad in (dict(lens=[79, 33, 97]), dict(lens=[-1, 33, 96]), dict(state=[6, 4]), dict(state=[8, 0])):
        r = int8.evict(tables, weights, bad.get("lens", [79, 33, 96]), 16, 3, 1, 1, np.arange(8),
                       bad.get("state", [6, 3]), [0, 0, 0])
        assert r[-1] and np.array_equal(r[0], tables) and np.array_equal(r[3], np.arange(8))


def test_norm_rope_against_a_rotation_matrix():
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((3, 2, 64)), rng.standard_normal(64)
    a = rng.uniform(0, 6, (9, 16))
    table = np.concatenate([np.cos(a), np.sin(a)], 1)
    pos = [8, 0, 3]
    plain = int8.norm_rope(x, w, 1e-3, None, pos, False)
    assert np.allclose(plain, x * w / np.sqrt((x ** 2).sum(-1, keepdims=True) / 64 + 1e-3))
    for inter in (False, True):
        got = int8.norm_rope(x, w, 1e-3, table, pos, inter)
        assert np.array_equal(got[..., 32:], plain[..., 32:])
        m = np.zeros((3, 64, 64)) + np.eye(64)
        for t, p in enumerate(pos):
            for i in range(16):
                u, v = (2 * i, 2 * i + 1) if inter else (i, i + 16)
                m[t][[u, u, v, v], [u, v, u, v]] = np.cos(a[p, i]), -np.sin(a[p, i]), np.sin(a[p, i]), np.cos(a[p, i])
        assert np.allclose(got, np.einsum("tij,thj->thi", m, plain))


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

P = ctypes.c_void_p(256)
at = ctypes.c_void_p


def far(i):
    """A buffer's address, away from the others'."""
    return ctypes.c_void_p(i << 24)


def desc(**kw):
    d = dict(num_blocks=16, block_size=16, num_kv_heads=2, head_size=64, dtype=pa.PA_INT8)
    d.update(kw)
    return pa.CacheDesc(**d)


def write_call(d=None, **kw):
    d = desc() if d is None else d
    return pa.lib.pa_reshape_and_cache_int8(
        kw.get("cache", far(1)), ctypes.byref(d), kw.get("key", far(2)), kw.get("value", far(3)),
        kw.get("dtype", pa.PA_BF16), kw.get("ks", 128), kw.get("vs", 128), kw.get("slots", P),
        kw.get("n", 4), None)


def gather_call(d=None, **kw):
    d = desc() if d is None else d
    return pa.lib.pa_gather_cache_int8(
        kw.get("key", far(2)), kw.get("value", far(3)), kw.get("dtype", pa.PA_BF16),
        kw.get("cache", far(1)), ctypes.byref(d), kw.get("slots", P), kw.get("n", 4), None)


def decode_call(d=None, **kw):
    d = desc() if d is None else d
    g = kw.get
    return pa.lib.pa_decode_int8(
        g("out", far(2)), g("query", far(3)), g("dtype", pa.PA_BF16), g("qs", 14 * 64),
        g("cache", far(1)), ctypes.byref(d), g("tables", far(4)), g("mb", 4), g("lens", far(5)), g("s", 2),
        g("heads", 14), g("scale", 0.125), g("before", None), g("after", None), g("decay", 1.0),
        g("ws", far(64)), g("ws_bytes", 1 << 30), None)


@pytest.mark.parametrize("call", [write_call, gather_call, decode_call])
@pytest.mark.parametrize("bad", [dict(dtype=pa.PA_BF16), dict(dtype=pa.PA_FP4), dict(block_size=4),
                                 dict(block_size=24), dict(block_size=512), dict(num_blocks=0),
                                 dict(num_kv_heads=0), dict(head_size=0)])
def test_bad_pools_are_refused(call, bad):
    assert call(desc(**bad)) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [write_call, gather_call, decode_call])
def test_bad_arguments_are_refused(call):
    assert call(desc(head_size=96)) == pa.PA_ERR_UNSUPPORTED
    assert call(desc(num_kv_heads=65535, block_size=256, head_size=256)) == pa.PA_ERR_UNSUPPORTED
    for bad in (pa.PA_FP4, pa.PA_INT8, 7):
        assert call(dtype=bad) == pa.PA_ERR_INVALID_ARG
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
        assert decode_call(decay=bad) == pa.PA_ERR_INVALID_ARG
    assert decode_call(qs=13 * 64) == pa.PA_ERR_INVALID_ARG
    assert decode_call(qs=14 * 64 + 4) == pa.PA_ERR_INVALID_ARG
    for name in ("out", "query", "ws"):
        assert decode_call(**{name: None}) == pa.PA_ERR_INVALID_ARG
        assert decode_call(**{name: ctypes.c_void_p(264)}) == pa.PA_ERR_INVALID_ARG
    for name in ("tables", "lens"):
        assert decode_call(**{name: None}) == pa.PA_ERR_INVALID_ARG
    assert decode_call(before=far(7)) == pa.PA_ERR_INVALID_ARG  # nowhere to put the sums
    for name in ("before", "after"):
        assert decode_call(**dict(dict(before=far(7), after=far(8)), **{name: at((9 << 24) + 2)})) == \
            pa.PA_ERR_INVALID_ARG


def test_overlapping_buffers_are_refused():
    # rows of 256 bytes and more, a pool of 16 blocks, four slots
    row, pool, slots = 4 * 256, 16 * 2 * 2 * 16 * 65, 4 * 8
    for name, size, step in (("key", row, 16), ("value", row, 16), ("slots", slots, 8)):
        for x in ((1 << 24) - size + step, 1 << 24, (1 << 24) + pool - 16):
            assert write_call(**{name: at(x)}) == pa.PA_ERR_INVALID_ARG, name
            if name != "slots":
                assert gather_call(**{name: at(x)}) == pa.PA_ERR_INVALID_ARG, name
    assert write_call(ks=2000, key=at((1 << 24) - 2 * (3 * 2000 + 128) + 16)) == pa.PA_ERR_INVALID_ARG
    for x in (-(row - 16), 0, row - 16):
        assert gather_call(key=at((3 << 24) + x)) == pa.PA_ERR_INVALID_ARG
    for out in (2, 3):
        for x in ((out << 24) - slots + 8, out << 24, (out << 24) + row - 8):
            assert gather_call(slots=at(x)) == pa.PA_ERR_INVALID_ARG
    # two rows of 14 heads of 64, tables and weights of two rows of four, two lengths
    size = 2 * 14 * 64 * 2
    for name, i, other, step in (("cache", 1, pool, 16), ("tables", 4, 32, 4), ("lens", 5, 8, 4),
                                 ("query", 3, size, 16)):
        for x in ((2 << 24) - other + step, 2 << 24, (2 << 24) + size - 16):
            if name not in ("cache", "query") or x % 16 == 0:
                assert decode_call(**{name: at(x)}) == pa.PA_ERR_INVALID_ARG, name
        for x in ((i << 24) - 32 + step, (i << 24) + other - step):
            if x % 4 == 0:
                assert decode_call(after=at(x)) == pa.PA_ERR_INVALID_ARG, name
    assert decode_call(after=far(2)) == pa.PA_ERR_INVALID_ARG
    for x in (-28, -4, 4, 28):                       # neither in place nor apart
        assert decode_call(before=far(7), after=at((7 << 24) + x)) == pa.PA_ERR_INVALID_ARG


def test_other_calls_refuse_an_8_bit_pool():
    d = desc()
    assert pa.lib.pa_reshape_and_cache(P, ctypes.byref(d), P, P, P, 4, None) == pa.PA_ERR_INVALID_ARG
    assert pa.lib.pa_decode(P, P, P, ctypes.byref(d), P, 4, P, 2, 14, 0.125, 64, 0, P, 1 << 20,
                            None) == pa.PA_ERR_INVALID_ARG
    assert pa.lib.pa_reshape_and_cache_fp4(far(1), ctypes.byref(d), far(2), far(3), pa.PA_BF16, 128, 128, P, 4,
                                           1.0, 1.0, None) == pa.PA_ERR_INVALID_ARG
    for other in (pa.PA_BF16, pa.PA_FP4):
        b = desc(dtype=other)
        assert pa.lib.pa_swap_blocks(P, ctypes.byref(d), P, ctypes.byref(b), P, 1,
                                     None) == pa.PA_ERR_INVALID_ARG
    assert pa.lib.pa_copy_blocks(P, ctypes.byref(desc(block_size=4)), P, 1,
                                 None) == pa.PA_ERR_INVALID_ARG


def evict_call(**kw):
    g = kw.get
    return pa.lib.pa_evict_blocks(
        g("tables", far(1)), g("weights", far(2)), g("mb", 4), g("lens", far(3)), g("n", 2), g("bs", 16),
        g("most", 3), g("first", 1), g("last", 1), g("ring", far(4)), g("cap", 5), g("state", far(5)),
        g("gone", far(6)), g("tables_out", far(7)), g("weights_out", far(8)), g("lens_out", far(9)),
        g("state_out", far(10)), g("gone_out", far(11)), None)


def test_evict_refusals():
    bad = [dict(n=-1), dict(n=8193), dict(mb=0), dict(mb=49153), dict(bs=12), dict(bs=0), dict(bs=512),
           dict(first=-1), dict(last=0), dict(most=1), dict(first=3), dict(first=(1 << 31) - 1), dict(most=-5),
           dict(ring=None), dict(state=None), dict(state_out=None), dict(cap=0), dict(cap=-1),
           dict(cap=(1 << 30) + 1), dict(ring=None, state=None, state_out=None),
           dict(gone=None), dict(gone_out=None)]
    bad += [{n: None} for n in ("tables", "weights", "lens", "tables_out", "weights_out", "lens_out")]
    bad += [{n: at((20 << 24) + 2)} for n in ("tables", "weights", "lens", "ring", "state", "gone", "tables_out",
                                              "weights_out", "lens_out", "state_out", "gone_out")]
    for kw in bad:
        assert evict_call(**kw) == pa.PA_ERR_INVALID_ARG, kw


def test_evict_overlaps_are_refused():
    # two rows of four entries, two lengths and counts, a ring of five
    sizes = dict(tables=32, weights=32, lens=8, ring=20, state=8, gone=8, tables_out=32, weights_out=32, lens_out=8,
                 state_out=8, gone_out=8)
    where = dict(tables=1, weights=2, lens=3, ring=4, state=5, gone=6, tables_out=7, weights_out=8, lens_out=9,
                 state_out=10, gone_out=11)
    for a in ("ring", "tables_out", "weights_out", "lens_out", "state_out", "gone_out"):
        for b in sizes:
            if b == a:
                continue
            for x in ((where[b] << 24) - sizes[a] + 4, (where[b] << 24) + sizes[b] - 4):
                assert evict_call(**{a: at(x)}) == pa.PA_ERR_INVALID_ARG, (a, b)
            if a != b + "_out":
                assert evict_call(**{a: far(where[b])}) == pa.PA_ERR_INVALID_ARG, (a, b)


def rope_call(**kw):
    g = kw.get
    a = pa.NormRopeArgs()
    for name, i in (("query_out", 1), ("key_out", 2), ("query", 3), ("key", 4), ("query_weight", 5),
                    ("key_weight", 6), ("cos_sin", 7), ("positions", 8), ("position_offsets", 9)):
        setattr(a, name, g(name, far(i)))
    a.query_out_stride = a.query_stride = 4 * 64
    a.key_out_stride = a.key_stride = 2 * 64
    a.eps, a.dtype, a.num_tokens, a.num_heads, a.num_kv_heads, a.head_size = 1e-6, pa.PA_BF16, 3, 4, 2, 64
    a.rotary_dim, a.max_position, a.interleaved = 64, 100, 0
    for name, _ in a._fields_[4:]:
        if name in kw and not name.endswith(("weight", "sin", "positions", "offsets")):
            setattr(a, name, kw[name])
    return pa.lib.pa_norm_rope(ctypes.byref(a), None)


def test_norm_rope_refusals():
    assert pa.lib.pa_norm_rope(None, None) == pa.PA_ERR_INVALID_ARG
    bad = [dict(dtype=pa.PA_INT8), dict(dtype=9), dict(num_tokens=-1), dict(num_heads=0), dict(num_kv_heads=0),
           dict(head_size=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(interleaved=2),
           dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=80), dict(rotary_dim=-16), dict(max_position=0),
           dict(cos_sin=None), dict(positions=None)]
    bad += [{n: None} for n in ("query_out", "key_out", "query", "key")]
    bad += [{n: at((20 << 24) + 8)} for n in ("query_out", "key_out", "query", "key", "query_weight", "key_weight",
                                              "cos_sin")]
    bad += [{n: at((20 << 24) + 2)} for n in ("positions", "position_offsets")]
    bad += [{n: v} for n in ("query_stride", "query_out_stride") for v in (248, 0, -256, 260)]
    bad += [{n: v} for n in ("key_stride", "key_out_stride") for v in (120, 132)]
    for kw in bad:
        assert rope_call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert rope_call(head_size=96) == pa.PA_ERR_UNSUPPORTED
    assert rope_call(num_heads=1 << 21) == pa.PA_ERR_UNSUPPORTED
    assert rope_call(num_tokens=0, query=None, key=None, query_out=None, key_out=None, positions=None) == pa.PA_OK


def test_norm_rope_overlaps_are_refused():
    # three rows of 512 (queries) and 256 bytes (keys)
    q, k = 3 * 512, 3 * 256
    for name, i, size in (("query", 3, q), ("key", 4, k), ("query_weight", 5, 128), ("key_weight", 6, 128),
                          ("cos_sin", 7, 100 * 64 * 4), ("positions", 8, 12), ("position_offsets", 9, 12)):
        for out, mine in (("query_out", q), ("key_out", k)):
            for x in ((i << 24) - mine + 16, (i << 24) + (size - 4) // 16 * 16):
                assert rope_call(**{out: at(x)}) == pa.PA_ERR_INVALID_ARG, (name, out)
    assert rope_call(query_out=far(4)) == pa.PA_ERR_INVALID_ARG
    assert rope_call(query_out=far(3), query_out_stride=512) == pa.PA_ERR_INVALID_ARG  # not in place
    # rows of a fused projection: keys behind the queries, or into them
    fused = dict(query_stride=1024, query_out_stride=1024, key_stride=1024, key_out_stride=1024)
    base = 30 << 24
    for off in (496, 2048 - 240, -16):
        assert rope_call(query=at(base), query_out=at(base), key=at(base + off), key_out=at(base + off),
                         **fused) == pa.PA_ERR_INVALID_ARG, off


def test_python_refusals():
    c = torch.zeros((4, 2, 2, 16 * 65), dtype=torch.int8)
    d = pa.int8_cache_desc(c)
    assert (d.num_blocks, d.block_size, d.num_kv_heads, d.head_size, d.dtype) == (4, 16, 2, 64, pa.PA_INT8)
    assert pa.alloc_int8_cache(4, 16, 2, 64, device="cpu").shape == c.shape
    for block in (-16, 0, 4, 7, 24, 512):
        with pytest.raises(ValueError):
            pa.alloc_int8_cache(4, block, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        pa.int8_cache_desc(c.view(torch.uint8))
    with pytest.raises(ValueError):
        pa.int8_cache_desc(c[..., :100].contiguous())
    with pytest.raises(ValueError):
        pa.int8_cache_desc(c[..., :16].contiguous())
    with pytest.raises(ValueError):
        pa.int8_cache_desc(c[..., ::2])
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):                      # host tensors
        pa.pa_reshape_and_cache_int8(c, k, k, s)
    with pytest.raises(TypeError):
        pa.pa_reshape_and_cache_int8(c, k, k.float(), s)
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache_int8(c, k, k[:2], s)
    with pytest.raises(ValueError):
        pa.pa_gather_cache_int8(k[:, :1], k[:, :1], c, s)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    w = torch.zeros((2, 3))
    with pytest.raises(ValueError):
        pa.pa_decode_int8(q, q, c, t[:1], n, 1.0, s)
    with pytest.raises(TypeError):
        pa.pa_decode_int8(q.float(), q, c, t, n, 1.0, s)
    with pytest.raises(ValueError):
        pa.pa_decode_int8(q, q, c, t, n, 1.0, s)         # host tensors
    for bad in (dict(tables=t[:1]), dict(weights=w[:, :2]), dict(lens=n[:1]), dict(ring=n), dict(state=n),
                dict(state_out=n), dict(gone_out=n), dict()):   # the last: host tensors
        with pytest.raises(ValueError):
            pa.pa_evict_blocks(bad.get("tables", t), bad.get("weights", w), bad.get("lens", n), 16, 3,
                               free_blocks=bad.get("ring"), free_state=bad.get("state"),
                               free_state_out=bad.get("state_out"), evicted_tokens_out=bad.get("gone_out"))
    p = n.clone()
    rope = lambda **kw: pa.pa_norm_rope(kw.get("qo", q), kw.get("ko", q[:, :2]), q, kw.get("k", q[:, :2]), None,
                                        None, kw.get("cs", torch.zeros((9, 64))), kw.get("p", p),
                                        position_offsets=kw.get("off"))
    for bad in (dict(qo=q[:, :2]), dict(k=q[:1, :2]), dict(ko=q), dict(p=p[:1]), dict(off=p[:1]), dict()):
        with pytest.raises(ValueError):
            rope(**bad)
    with pytest.raises(TypeError):
        rope(qo=q.float())


def test_sizes_past_32_bits_are_refused():
    """Not cut to 32 bits, where they could pass for small ones."""
    meta = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="meta")
    big = (1 << 32) + 8
    cache, lens = meta(4, 2, 2, 16 * 65, dtype=torch.int8), meta(1)
    q = meta(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="past 2"):
        pa.pa_decode_int8(q, q, cache, meta(1, big), lens, 1.0, lens)
    with pytest.raises(ValueError, match="past 2"):
        pa.pa_decode_int8_workspace_size(pa.int8_cache_desc(cache), 4, meta(1, big))
    rows, slots = meta(big, 2, 64, dtype=torch.bfloat16), meta(big, dtype=torch.int64)
    with pytest.raises(ValueError, match="past 2"):
        pa.pa_reshape_and_cache_int8(cache, rows, rows, slots)
    with pytest.raises(ValueError, match="past 2"):
        pa.pa_gather_cache_int8(rows, rows, cache, slots)
    for kw in (dict(tables=meta(1, big)), dict(size=big), dict(most=big), dict(first=big), dict(last=big),
               dict(ring=meta(big))):
        t, ring = kw.get("tables", meta(1, 4)), kw.get("ring")
        with pytest.raises(ValueError, match="past 2"):
            pa.pa_evict_blocks(t, meta(*t.shape, dtype=torch.float32), lens, kw.get("size", 16), kw.get("most", 3),
                               kw.get("first", 1), kw.get("last", 1), free_blocks=ring,
                               free_state=None if ring is None else meta(2))
    with pytest.raises(ValueError, match="past 2"):
        pa.pa_norm_rope(rows, rows, rows, rows, None, None, None, meta(big))


def test_numbers_outside_32_bits_are_refused():
    """Negative ones that would be cut to a small positive number, and counts of heads."""
    meta = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="meta")
    t, w, lens = meta(1, 4), meta(1, 4, dtype=torch.float32), meta(1)
    small = -(1 << 32)
    for kw in (dict(size=small + 16), dict(most=small + 3), dict(first=small + 1), dict(last=small + 1),
               dict(first=-(1 << 31) - 1)):
        with pytest.raises(ValueError, match="outside 32 bits"):
            pa.pa_evict_blocks(t, w, lens, kw.get("size", 16), kw.get("most", 3), kw.get("first", 1),
                               kw.get("last", 1))
    for kw in (dict(size=small + 16), dict(blocks=small + 8)):
        with pytest.raises(ValueError, match="outside 32 bits"):
            pa.pa_extend_tables(t, lens, lens, kw.get("size", 16), kw.get("blocks", 8), meta(1, dtype=torch.int64))
    int8_desc, fp4_desc = desc(), pa.CacheDesc(8, 16, 2, 64, pa.PA_FP4)
    for heads in ((1 << 32) + 4, small + 4):
        with pytest.raises(ValueError, match="past 2|outside 32 bits"):
            pa.pa_decode_int8_workspace_size(int8_desc, heads)
        with pytest.raises(ValueError, match="past 2|outside 32 bits"):
            pa.pa_decode_fp4_workspace_size(fp4_desc, heads)


def test_workspace_size_refusals():
    out = ctypes.c_size_t()
    call = lambda d, h, s=0, b=0: pa.lib.pa_decode_int8_workspace_size(ctypes.byref(d), h, s, b, ctypes.byref(out))
    assert call(desc(dtype=pa.PA_FP4), 4) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 3) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 0) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 4, -1) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 4, 65536) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 4, 1, -1) == pa.PA_ERR_INVALID_ARG
    assert call(desc(), 34) == pa.PA_ERR_UNSUPPORTED
    # more entries than 32 bits count, whose bytes 64 bits might not
    for s, b in ((65535, (1 << 31) - 1), (3, (1 << 31) - 1), (65535, 65538)):
        assert call(desc(), 4, s, b) == pa.PA_ERR_UNSUPPORTED
    heads = desc(num_kv_heads=65535, head_size=64, block_size=8)
    assert call(heads, 16 * 65535, 65535, (1 << 31) - 1) == pa.PA_ERR_UNSUPPORTED
    assert decode_call(s=65535, mb=65538, after=far(90), ws_bytes=1 << 62, out=far(70)) == pa.PA_ERR_UNSUPPORTED
    assert call(desc(head_size=32), 4) == pa.PA_ERR_UNSUPPORTED
