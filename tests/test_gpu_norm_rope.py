"""Norms of queries and keys with the rotation on the GPU against the binary64 oracle, and
the whole decode step over an 8-bit pool: eviction, tables, norms and rotation, write, attention."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_78_gb300 as pa
from int8_util import TORCH, assert_decode, assert_weights, host, rounded
from oracle import fp4, int8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    pa.pa_get_device_error()
    yield


def dev(a, dtype=None):
    t = a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))
    return t.cuda() if dtype is None else t.to(dtype).cuda()


def table(positions, rotary, seed=0):
    rate = 10000.0 ** (-np.arange(rotary // 2) * 2 / rotary)
    a = np.arange(positions)[:, None] * rate
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rope_bound(x, weight, eps, cos_sin, positions, interleaved, dtype):
    """The norm: a sum of squares, 16 in a row and 4 over lanes at the most (2^-24 each, halved by the
    root: 10), eps (halved), the root (2 last places: 2.2), two products: 15 * 2^-24.  The rotation: a
    product and a sum each of |u c| + |v s|: 3 * 2^-24.  One rounding to the type, half a step."""
    if cos_sin is None:
        near = np.abs(int8.norm_rope(x, weight, eps, None, positions, interleaved))
    else:
        # |u c| + |v s| is what a rotation by |c|, -|s| of |x| gives for the first of a pair, by |s| for
        # the second
        half = cos_sin.shape[1] // 2
        a = np.abs(int8.norm_rope(x, weight, eps, None, positions, interleaved))
        cs = np.abs(cos_sin[np.asarray(positions)])[:, None]
        near = a.copy()
        for i in range(half):
            u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = cs[..., i], cs[..., half + i]
            near[..., u], near[..., v] = a[..., u] * c + a[..., v] * s, a[..., v] * c + a[..., u] * s
    return near, 18 * 2.0 ** -24 * near


def assert_rope(got, x, weight, eps, cos_sin, positions, interleaved, dtype, what=""):
    x, w = host(x), None if weight is None else host(weight)
    ref = int8.norm_rope(x, w, eps, cos_sin, positions, interleaved)
    _, bound = rope_bound(x, w, eps, cos_sin, positions, interleaved, dtype)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    err = np.abs(host(got) - ref)
    assert (err <= bound + half * (np.abs(ref) + bound) + 1e-40).all(), what


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("head,rotary,heads,hkv,n", [
    (64, 64, 14, 2, 1), (64, 32, 3, 1, 33), (128, 128, 32, 8, 7), (128, 64, 5, 5, 100), (256, 256, 16, 2, 9),
    (256, 32, 1, 1, 2), (128, 16, 8, 8, 3), (64, 0, 4, 4, 5), (128, 0, 6, 2, 300), (128, 112, 4, 2, 21),
    (64, 48, 40, 8, 2000), (128, 128, 4, 1, 40001)])
def test_norm_rope(head, rotary, heads, hkv, n, dtype, interleaved):
    rng = np.random.default_rng(head + n)
    far = 5000
    cs = table(far, rotary) if rotary else None
    q, k = (rounded(np.exp(rng.standard_normal((n, h, 1))) * rng.standard_normal((n, h, head)), dtype)
            for h in (heads, hkv))
    qw, kw = (rounded(rng.standard_normal(head), dtype) for _ in range(2))
    pos, off = rng.integers(0, far // 2, n), rng.integers(-3, far // 2, n)
    off = np.maximum(off, -pos)
    qo, ko = torch.full_like(dev(q), 7), torch.full_like(dev(k), 7)
    pa.pa_norm_rope(qo, ko, dev(q), dev(k), dev(qw), dev(kw), None if cs is None else dev(cs), dev(pos, torch.int32),
                    1e-5, interleaved, dev(off, torch.int32))
    some = slice(None) if n < 3000 else np.r_[0:100, n // 2:n // 2 + 100, n - 100:n]
    at = (pos + off)[some]
    assert_rope(qo[some], q[some], qw, 1e-5, cs, at, interleaved, dtype)
    assert_rope(ko[some], k[some], kw, 1e-5, cs, at, interleaved, dtype)
    # without weights and offsets, in place, slices of one projection
    wide = torch.full((n, (heads + 2 * hkv) * head + 16), 3.0, dtype=TORCH[dtype], device="cuda")
    qs = wide[:, :heads * head].unflatten(1, (heads, head))
    ks = wide[:, heads * head:(heads + hkv) * head].unflatten(1, (hkv, head))
    qs.copy_(dev(q)), ks.copy_(dev(k))
    pa.pa_norm_rope(qs, ks, qs, ks, None, None, None if cs is None else dev(cs), dev(pos, torch.int32), 0.5, interleaved)
    assert_rope(qs[some], q[some], None, 0.5, cs, pos[some], interleaved, dtype)
    assert_rope(ks[some], k[some], None, 0.5, cs, pos[some], interleaved, dtype)
    assert (wide[:, (heads + hkv) * head:] == 3).all()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("rotary", [0, 64])
def test_padding_and_positions_past_the_table(rotary):
    rng = np.random.default_rng(1)
    q, k = rounded(rng.standard_normal((7, 4, 64)), "bf16"), rounded(rng.standard_normal((7, 2, 64)), "bf16")
    cs = table(10, rotary) if rotary else None
    pos = np.array([0, -1, 9, 10, -(1 << 31), (1 << 31) - 1, 3])
    off = np.array([9, 5, 0, 0, 4, (1 << 31) - 1, -4])
    qo, ko = torch.full((9, 4, 64), 7, dtype=torch.bfloat16, device="cuda"), torch.full((9, 2, 64), 8, dtype=torch.bfloat16,
                                                                                        device="cuda")
    pa.pa_norm_rope(qo[:7], ko[:7], dev(q), dev(k), None, None, None if cs is None else dev(cs), dev(pos, torch.int32),
                    0.0, False, dev(off, torch.int32))
    assert pa.pa_get_device_error() == (pa.PA_DEVERR_POSITION if rotary else 0)
    live = [0, 2] if rotary else [0, 2, 3, 5, 6]
    dead = np.setdiff1d(np.arange(9), live)
    at = (pos + off)[live] if rotary else live
    assert_rope(qo[live], q[live], None, 0.0, cs, at, False, "bf16")
    assert_rope(ko[live], k[live], None, 0.0, cs, at, False, "bf16")
    assert (qo[dead] == 7).all() and (ko[dead] == 8).all()


def test_special_values():
    x = np.ones((6, 1, 64))
    x[0] = 0.0
    x[1, 0, 5] = np.nan
    x[2, 0, 5] = np.inf
    x[3] = 2.0 ** -60
    x[4] = 2.0 ** 55
    x[5] = 2.0 ** -140
    t = rounded(x, "fp32")
    out = [torch.empty_like(dev(t)) for _ in range(2)]
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    pa.pa_norm_rope(out[0], out[1], dev(t), dev(t), None, None, None, pos, 0.0)
    y = host(out[0])[:, 0]
    assert np.isnan(y[:2]).all() and np.isnan(y[2, 5]) and not y[2, :5].any()
    assert np.abs(y[3:5] - 1).max() < 1e-6
    pa.pa_norm_rope(out[0], out[1], dev(t), dev(t), None, None, None, pos, 1e-6)
    y = host(out[1])[:, 0]
    assert not y[0].any() and np.abs(y[5] - 2.0 ** -140 / 1e-3).max() < 2.0 ** -148


def test_far_strides_and_streams():
    """Rows gigabytes apart, and a call on another stream than the current one."""
    n, stride = 3, (1 << 30) + 8
    flat = torch.empty((n - 1) * stride + 6 * 64, dtype=torch.bfloat16, device="cuda")
    q, k = flat.as_strided((n, 4, 64), (stride, 64, 1)), flat.as_strided((n, 2, 64), (stride, 64, 1), 4 * 64)
    x = rounded(np.random.default_rng(3).standard_normal((n, 6, 64)), "bf16")
    q.copy_(dev(x[:, :4])), k.copy_(dev(x[:, 4:]))
    cs, s = table(9, 64), torch.cuda.Stream()
    torch.cuda.synchronize()
    pa.pa_norm_rope(q, k, q, k, None, None, dev(cs), dev(np.array([8, 0, 2]), torch.int32), 1e-6, stream=s)
    s.synchronize()
    assert_rope(q, x[:, :4], None, 1e-6, cs, [8, 0, 2], False, "bf16")
    assert_rope(k, x[:, 4:], None, 1e-6, cs, [8, 0, 2], False, "bf16")


# ---------------------------------------------------------------------------
# the step
# ---------------------------------------------------------------------------

class Shell:
    """What the bounds want to know of a batch."""

    def __init__(self, query, cache, tables, lens, scale, block, dtype):
        self.query, self.cache, self.tables, self.lens = query, cache, tables, lens
        self.scale, self.block, self.dtype = scale, block, dtype

    def reference(self):
        return int8.decode(host(self.query), self.cache, self.tables, self.lens, self.scale)


@pytest.mark.parametrize("dtype,heads,hkv,head,block", [("bf16", 8, 2, 128, 16), ("bf16", 5, 5, 64, 8),
                                                        ("fp32", 6, 2, 256, 16)])
def test_captured_step_serves_sequences_that_lose_blocks(dtype, heads, hkv, head, block):
    """evict -> tables -> norms and rotation -> write -> decode with weights, captured once and
    replayed for every step.  Each stage is checked against the oracle on what the device held before the
    step; a pool of few blocks suffices, as sequences keep at most four."""
    rng = np.random.default_rng(head)
    prompts, most = [3, block, 0, 4 * block - 1], 4
    blocks, width, steps = 18, 7, 4 * block + 3
    s, scale, far = len(prompts), head ** -0.5, 6 * block + 80
    i32 = lambda a: dev(np.asarray(a), torch.int32)
    cache = torch.randint(-128, 128, (blocks, hkv, block // 8, 16 * (head + 1)), dtype=torch.int8, device="cuda")
    tables, lens = torch.zeros((s, width), dtype=torch.int32, device="cuda"), i32([0] * s)
    ring, state = i32(rng.permutation(blocks)), i32([0, blocks])
    weights, gone = torch.zeros((s, width), device="cuda"), i32([0] * s)
    n = sum(prompts)
    slots0 = torch.empty(n, dtype=torch.int64, device="cuda")
    pa.pa_extend_tables(tables, lens, i32(prompts), block, blocks, slots0, free_blocks=ring, free_state=state)
    pk, pv = (rounded(rng.standard_normal((n, hkv, head)), dtype) for _ in range(2))
    pa.pa_reshape_and_cache_int8(cache, dev(pk), dev(pv), slots0)

    cs = table(far, head)
    one, csd = i32([1] * s), dev(cs)
    qw, kw = (rounded(1 + 0.2 * rng.standard_normal(head), dtype) for _ in range(2))
    qwd, kwd = dev(qw), dev(kw)
    slots = torch.empty(s, dtype=torch.int64, device="cuda")
    pos = torch.empty(s, dtype=torch.int32, device="cuda")
    qkv = torch.zeros((s, (heads + 2 * hkv) * head), dtype=TORCH[dtype], device="cuda")
    q, k, v = qkv.split([heads * head, hkv * head, hkv * head], dim=1)
    q, k, v = q.unflatten(1, (heads, head)), k.unflatten(1, (hkv, head)), v.unflatten(1, (hkv, head))
    qr = torch.empty((s, heads, head), dtype=TORCH[dtype], device="cuda")
    kr = torch.empty((s, hkv, head), dtype=TORCH[dtype], device="cuda")
    out = torch.empty_like(qr)
    ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(cache, heads, tables), "cuda")

    def step():
        pa.pa_evict_blocks(tables, weights, lens, block, most, 1, 1, ring, state, gone)
        pa.pa_extend_tables(tables, lens, one, block, blocks, slots, positions=pos, free_blocks=ring, free_state=state)
        pa.pa_norm_rope(qr, kr, q, k, qwd, kwd, csd, pos, 1e-6, position_offsets=gone)
        pa.pa_reshape_and_cache_int8(cache, kr, v, slots)
        pa.pa_decode_int8(out, qr, cache, tables, lens, scale, ws, block_weights=weights, decay=0.9)

    held = (tables, lens, ring, state, weights, gone, cache)
    saved = [t.clone() for t in held]
    step()                               # once outside, then put everything back
    torch.cuda.synchronize()
    for t, was in zip(held, saved):
        t.copy_(was)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    total = np.array(prompts)
    for i in range(steps):
        qkv.copy_(rounded(rng.standard_normal(tuple(qkv.shape)), dtype))
        t0, n0, r0, s0, w0, g0, c0 = (x.cpu().numpy().copy() for x in held)
        g.replay()
        t, w, n1, r, st, gn, refused = int8.evict(t0, w0, n0, block, most, 1, 1, r0, s0, g0)
        assert not refused
        t, n1, st, sl, ps, _, refused = fp4.extend_tables(t, n1, [1] * s, block, blocks, s, r, st)
        assert not refused
        total = total + 1
        assert np.array_equal(host(tables), t) and np.array_equal(host(lens), n1), i
        assert np.array_equal(host(slots), sl) and np.array_equal(host(pos), ps), i
        assert np.array_equal(host(gone), gn) and host(state).tolist() == list(st), i
        assert np.array_equal(host(ring), r) and np.array_equal(gn + n1, total), i
        assert (n1 <= most * block + 1).all()
        at = ps + gn
        assert_rope(qr, q, qw, 1e-6, cs, at, False, dtype, i)
        assert_rope(kr, k, kw, 1e-6, cs, at, False, dtype, i)
        int8.write(c0, host(kr), host(v), sl)
        b = Shell(qr.cpu(), cache.cpu().numpy(), t, n1, scale, block, dtype)
        live = np.concatenate([t[x, np.arange(y) // block] * block + np.arange(y) % block for x, y in enumerate(n1)])
        for x, y in zip(int8.read(b.cache, live), int8.read(c0, live)):
            assert np.array_equal(x, y), i
        ref = b.reference()
        assert_decode(out, b, "step %d" % i, ref)
        assert_weights(weights, b, w, 0.9, w, "step %d" % i, ref)
    assert (total > most * block).all() and pa.pa_get_device_error() == 0


def test_a_row_that_a_new_sequence_takes_begins_at_zero():
    """A captured step; both rows' sequences end, and others take the rows with weights and
    evicted tokens set to zero: every later step is what it is for the same sequences in rows that
    no other had before, bit for bit, evictions among it."""
    block, most, heads, hkv, head, width, blocks, s = 8, 4, 4, 2, 64, 6, 24, 2
    rng = np.random.default_rng(31)
    i32 = lambda a: dev(np.asarray(a), torch.int32)
    cs, one = dev(table(200, head)), i32([1] * s)
    qkv = torch.zeros((s, heads + 2 * hkv, head), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv.split([heads, hkv, hkv], dim=1)

    class Server:
        def __init__(self):
            self.cache = pa.alloc_int8_cache(blocks, block, hkv, head)
            self.tables = torch.zeros((s, width), dtype=torch.int32, device="cuda")
            self.lens, self.gone, self.pos = i32([0] * s), i32([0] * s), i32([0] * s)
            self.ring, self.state = i32(np.arange(blocks)), i32([0, blocks])
            self.weights = torch.zeros((s, width), device="cuda")
            self.slots = torch.empty(s, dtype=torch.int64, device="cuda")
            self.q, self.k = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
            self.out = torch.empty_like(self.q)
            self.ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(self.cache, heads, self.tables), "cuda")
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.step()

        def step(self):
            pa.pa_evict_blocks(self.tables, self.weights, self.lens, block, most, 1, 1, self.ring, self.state,
                               self.gone)
            pa.pa_extend_tables(self.tables, self.lens, one, block, blocks, self.slots, positions=self.pos,
                                free_blocks=self.ring, free_state=self.state)
            pa.pa_norm_rope(self.q, self.k, q, k, None, None, cs, self.pos, position_offsets=self.gone)
            pa.pa_reshape_and_cache_int8(self.cache, self.k, v, self.slots)
            pa.pa_decode_int8(self.out, self.q, self.cache, self.tables, self.lens, head ** -0.5, self.ws,
                              block_weights=self.weights, decay=0.9)

        def begin(self, row):
            """The row's blocks go back to the ring; a new sequence has none."""
            n = -(-int(self.lens[row]) // block)
            front, count = self.state.tolist()
            for i in range(n):
                self.ring[(front + count + i) % blocks] = self.tables[row, i]
            self.state[1] += n
            self.lens[row], self.gone[row], self.weights[row] = 0, 0, 0.0

        def seen(self):
            lens = self.lens.tolist()
            return lens, self.gone.tolist(), [self.weights[r, :-(-n // block)].tolist() for r, n in enumerate(lens)]

    rows = lambda: rounded(rng.standard_normal(tuple(qkv.shape)), "bf16")
    old, fresh = Server(), Server()
    for _ in range(block * most + 2 * block + 3):
        qkv.copy_(rows())
        old.graph.replay()
    assert min(old.gone.tolist()) > 0 and (old.weights[:, :most] > 0).all()
    old.begin(0), old.begin(1)
    assert old.state.tolist()[1] == blocks
    for i in range(block * most + 3 * block + 1):             # long enough to lose blocks again
        qkv.copy_(rows())
        old.graph.replay(), fresh.graph.replay()
        assert torch.equal(old.out, fresh.out) and old.seen() == fresh.seen(), i
    assert min(old.gone.tolist()) > 0 and pa.pa_get_device_error() == 0


FIRST_CALLS = """
import torch
import paged_kv_cache_78_gb300 as pa
t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache = pa.alloc_int8_cache(6, 8, 1, 64)
kv = torch.full((2, 1, 64), 6.0, device="cuda")
out, back, kn = (torch.empty((2, 1, 64), device="cuda") for _ in range(3))
tables, lens, state = t(1, 2, 3, 4).view(2, 2), t(1, 9), t(0, 2)
slots = torch.tensor([8, 32], device="cuda")
weights, gone, ring, pos = torch.ones((2, 2), device="cuda"), t(0, 0), t(5, 0, 0, 0), t(0, 0)
ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(cache, 1, tables), "cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pa.pa_evict_blocks(tables, weights, lens, 8, 1, 0, 1, ring, state, gone)
    pa.pa_norm_rope(out, kn, kv, kv, None, None, None, pos, 0.0)
    pa.pa_reshape_and_cache_int8(cache, kn, kv, slots)
    pa.pa_gather_cache_int8(back, out, cache, slots)
    pa.pa_decode_int8(out, kv, cache, tables, lens, 1.0, ws, block_weights=weights)
g.replay()
assert lens.tolist() == [1, 1] and gone.tolist() == [0, 8] and state.tolist() == [0, 3]
assert tables.tolist() == [[1, 2], [4, 3]] and ring[2] == 3 and weights.tolist() == [[2, 1], [2, 0]]
assert (back - 1).abs().max() < 1e-6 and (out - 6).abs().max() < 1e-5
print("captured")
"""


def test_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True,
                       timeout=280)
    assert r.returncode == 0 and r.stdout.split()[-1] == "captured", r.stderr


def test_calls_take_numpy_scalars():
    c = pa.alloc_int8_cache(np.int64(6), np.int64(8), np.int32(1), np.int64(64))
    kv = torch.ones((1, 1, 64), device="cuda")
    out, t, n = torch.empty_like(kv), torch.zeros((1, 2), dtype=torch.int32, device="cuda"), dev(np.array([1]), torch.int32)
    w = torch.zeros((1, 2), device="cuda")
    pa.pa_reshape_and_cache_int8(c, kv, kv, torch.zeros(1, dtype=torch.int64, device="cuda"))
    ws = pa.alloc_workspace(pa.pa_decode_int8_workspace_size(c, np.int64(1), t), "cuda")
    pa.pa_decode_int8(out, kv, c, t, n, np.float32(1), ws, block_weights=w, decay=np.float64(1))
    pa.pa_evict_blocks(t, w, n, np.int64(8), np.int64(2), np.int32(1), np.int64(1))
    pa.pa_norm_rope(out, kv, out, kv, None, None, None, n, np.float64(0), np.bool_(True))
    assert torch.equal(w, torch.tensor([[1.0, 0.0]], device="cuda")) and (out - 1).abs().max() < 1e-6
