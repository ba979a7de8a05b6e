"""The 4-bit paged cache's operators, as measured work: the same calls in their
plain form (elementary torch operations, 32 bits or more) and, where `own` is
true, through this repository's entry points.

A 4-bit cache holds keys and values as e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6
and their negatives) with one e4m3 scale per 16 elements of a head, in a
uint8 tensor [num_blocks, num_kv_heads, block_size / 8, 9 * head_size].  The
last axis is a tile of eight tokens:
    [8 tokens][head_size / 2]          key codes, even element in the low nibble
    [head_size / 16][8 tokens][8]      value codes, by groups of 16 elements
    [8 tokens][head_size / 16]         key scales
    [head_size / 16][8 tokens]         value scales
The value that a code stands for is code * scale * tensor scale (a power of
two per cache, one for the keys and one for the values).

Kinds of cases: "tables" (block tables, slot map and positions from request
lengths), "write" (new tokens quantised into the cache, and read back),
"gather" (cached tokens read back), "decode" (one query token per sequence)
and "step" (the three of a decode step in a row).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LARGEST_BYTES = 330_000_000  # of a drawn case: the largest listed one's


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a serving step's bookkeeping: every running request gets one token
        {"name": "tables_decode", "kind": "tables", "requests": 256, "context": "uniform:1:8192",
         "new": "fixed:1", "block": 16, "seed": 11},
        # prompts admitted and chunks continued in one step, some requests idle
        {"name": "tables_prefill", "kind": "tables", "requests": 500, "context": "uniform:0:4096",
         "new": "uniform:0:500", "block": 16, "seed": 12},
        # the newest tokens of a decode batch
        {"name": "write_decode", "kind": "write", "tokens": 64, "kv_heads": 2, "head": 64,
         "block": 16, "dtype": "bf16", "key_scale": 1.0, "value_scale": 0.25, "seed": 21},
        # a prompt chunk as a slice of the fused projection's output
        {"name": "write_prefill", "kind": "write", "tokens": 16381, "kv_heads": 8, "head": 128,
         "block": 16, "dtype": "bf16", "key_scale": 2.0, "value_scale": 0.5, "seed": 22},
        # a cached prefix of a few hundred tokens read back in fp32
        {"name": "gather_prefix", "kind": "gather", "tokens": 777, "kv_heads": 4, "head": 64,
         "block": 8, "dtype": "fp32", "key_scale": 1.0, "value_scale": 1.0, "seed": 31},
        # a long cached context read back for a prompt chunk's attention
        {"name": "gather_context", "kind": "gather", "tokens": 65536, "kv_heads": 8, "head": 128,
         "block": 16, "dtype": "bf16", "key_scale": 1.0, "value_scale": 0.5, "seed": 32},
        # the smallest batch: a few short sequences, latency
        {"name": "decode_tiny", "kind": "decode", "lens": "list:7,16,33,100", "heads": 4,
         "kv_heads": 4, "head": 64, "block": 8, "dtype": "bf16", "seed": 41},
        # grouped queries, ragged lengths
        {"name": "decode_gqa", "kind": "decode", "lens": "uniform:0:2048*64", "heads": 14,
         "kv_heads": 2, "head": 64, "block": 16, "dtype": "bf16", "seed": 42},
        # one query head per KV head, ragged lengths
        {"name": "decode_mha", "kind": "decode", "lens": "uniform:1:2048*32", "heads": 40,
         "kv_heads": 40, "head": 128, "block": 32, "dtype": "bf16", "seed": 43},
        # long contexts, the bound on memory
        {"name": "decode_long", "kind": "decode", "lens": "fixed:32768*8", "heads": 32,
         "kv_heads": 8, "head": 128, "block": 16, "dtype": "bf16", "seed": 44},
        # very different lengths (one sequence still empty), wide heads, 32-bit queries
        {"name": "decode_mixed_fp32", "kind": "decode", "lens": "list:0,1,513,4097,40001",
         "heads": 16, "kv_heads": 2, "head": 256, "block": 16, "dtype": "fp32", "seed": 45},
        # a whole decode step: tables, write, attention
        {"name": "step_gqa", "kind": "step", "lens": "uniform:0:4095*128", "heads": 32,
         "kv_heads": 8, "head": 128, "block": 16, "dtype": "bf16", "seed": 51},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("tables", "write", "gather", "decode", "decode", "step"))
    seed = rng.randrange(1 << 30)
    block = rng.choice((8, 16, 16, 32, 64, 128, 256))
    if kind == "tables":
        requests = _log_int(rng, 1, 2000)
        most = max(1, min(2000, 250_000 // requests))
        return {"kind": kind, "requests": requests,
                "context": "uniform:0:%d" % _log_int(rng, 1, 16384),
                "new": rng.choice(("fixed:1", "uniform:0:%d" % _log_int(rng, 1, most))),
                "block": block, "seed": seed}
    head = rng.choice((64, 128, 128, 256))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if kind in ("write", "gather"):
        kv_heads = rng.choice((1, 2, 3, 4, 8, 16, 40))
        once = 2 * kv_heads * head * (2.5625 if dtype == "bf16" else 4.5625)
        most = max(2, min(65536, int(LARGEST_BYTES / once) // (1 if kind == "gather" else 2)))
        return {"kind": kind, "tokens": _log_int(rng, 1, most), "kv_heads": kv_heads, "head": head,
                "block": block, "dtype": dtype, "key_scale": rng.choice((0.5, 1.0, 4.0)),
                "value_scale": rng.choice((0.125, 1.0, 2.0)), "seed": seed}
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 8, 12, 16))
    seqs = _log_int(rng, 1, 256)
    row = kv_heads * head * 9 // 8
    most = max(1, min(131072, LARGEST_BYTES // 2 // (seqs * row)))
    longest = _log_int(rng, 1, most)
    lens = rng.choice(("uniform:%d:%d*%d" % (rng.choice((0, 1)), longest, seqs),
                       "fixed:%d*%d" % (longest, seqs)))
    return {"kind": kind, "lens": lens, "heads": kv_heads * group, "kv_heads": kv_heads,
            "head": head, "block": block, "dtype": dtype, "seed": seed}


def _numbers(spec, seed, count=None):
    """The whole numbers that "fixed:n*count", "uniform:lo:hi*count" or
    "list:a,b,..." stand for."""
    spec, _, times = spec.partition("*")
    how, _, rest = spec.partition(":")
    if how == "list":
        return np.array([int(v) for v in rest.split(",")], dtype=np.int64)
    count = int(times) if times else count
    if how == "fixed":
        return np.full(count, int(rest), dtype=np.int64)
    lo, hi = (int(v) for v in rest.split(":"))
    return np.random.default_rng(seed).integers(lo, hi, size=count, endpoint=True)


def _context_and_new(case):
    if case["kind"] == "tables":
        n = case["requests"]
        return (_numbers(case["context"], case["seed"], n), _numbers(case["new"], case["seed"] + 1, n))
    context = _numbers(case["lens"], case["seed"])
    return context, np.ones_like(context)


def work(case):
    kind = case["kind"]
    if kind == "tables":
        context, new = _context_and_new(case)
        blocks = int((-(-(context + new) // case["block"])).sum() - (-(-context // case["block"])).sum())
        tokens, n = int(new.sum()), len(new)
        # lengths and counts in, lengths and starts out, free ids in and table
        # entries out, slots and positions out
        return {"bytes": 16 * n + 8 * blocks + 12 * max(tokens, 1), "flops": 0}
    elem = 2 if case["dtype"] == "bf16" else 4
    if kind in ("write", "gather"):
        values = 2 * case["tokens"] * case["kv_heads"] * case["head"]
        once = values * elem + values * 9 // 16 + 8 * case["tokens"]
        return {"bytes": once * (2 if kind == "write" else 1), "flops": 0}
    lens = _numbers(case["lens"], case["seed"])
    tokens, seqs = int(lens.sum()) + (len(lens) if kind == "step" else 0), len(lens)
    heads, kv_heads, head = case["heads"], case["kv_heads"], case["head"]
    read = tokens * kv_heads * 2 * head * 9 // 16 + 4 * int((-(-lens // case["block"])).sum()) + 4 * seqs
    ends = 2 * seqs * heads * head * elem
    new = seqs * (2 * kv_heads * head * elem + 2 * kv_heads * head * 9 // 16 + 28) if kind == "step" else 0
    return {"bytes": read + ends + new, "flops": 4 * tokens * heads * head}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(shape, gen, device):
    return torch.randn(shape, generator=gen, device=device, dtype=torch.float32)


def _outliers(x):
    """A few channels an order larger than the others, as keys have them."""
    x[..., 3::37] *= 6.0
    return x


def _filled_cache(blocks, kv_heads, block, head, gen, device):
    """A pool of quantised normal keys and values."""
    cache = torch.empty((blocks, kv_heads, block // 8, 9 * head), dtype=torch.uint8, device=device)
    step = max(1, (1 << 24) // (kv_heads * block * head))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        k = _outliers(_normal((n, kv_heads, block // 8, 8, head), gen, device))
        v = _normal((n, kv_heads, block // 8, 8, head), gen, device)
        kc, ks = _quantise(k)
        vc, vs = _quantise(v)
        vc = vc.view(n, kv_heads, block // 8, 8, head // 16, 8).transpose(-3, -2)
        cache[b:b + n] = torch.cat([kc.flatten(3), vc.flatten(3), ks.flatten(3),
                                    vs.transpose(-2, -1).flatten(3)], dim=-1)
    return cache


def _tables(lens, block, extra, perm, width=None):
    """Block tables that take `perm` in order, and the ids that are left."""
    counts = -(-lens // block)
    width = int(max(1, (-(-(lens + extra) // block)).max())) if width is None else width
    tables = np.zeros((len(lens), width), dtype=np.int32)
    at = 0
    for r, c in enumerate(counts):
        tables[r, :c] = perm[at:at + c]
        at += int(c)
    return tables, perm[at:]


def _kill_dead_rows(cache, tables, lens, block, head):
    """NaN scales in the rows of last blocks past their sequences' ends: what
    earlier owners of the blocks may have left there."""
    kv_heads, tiles, size = cache.shape[1:]
    dead = [(int(tables[r, n // block]), t) for r, n in enumerate(int(x) for x in lens)
            for t in range(n % block, block) if n % block]
    if not dead:
        return
    d = torch.tensor(dead, dtype=torch.int64, device=cache.device)
    tile, row = d[:, 1] // 8, d[:, 1] % 8
    groups = torch.arange(head // 16, device=cache.device)
    heads = torch.arange(kv_heads, device=cache.device)
    base = ((d[:, 0, None] * kv_heads + heads) * tiles + tile[:, None]) * size
    flat = cache.view(-1)
    for at in (8 * head + row[:, None] * (head // 16) + groups,
               8 * head + head // 2 + groups * 8 + row[:, None]):
        flat[base[:, :, None] + at[:, None, :]] = 0x7F


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    kind, block = case["kind"], case["block"]

    def put(a, dtype):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(device)

    s = dict(case)
    if kind in ("tables", "step"):
        context, new = _context_and_new(case)
        blocks = int((-(-(context + new) // block)).sum()) + 7
        tables, left = _tables(context, block, new, rng.permutation(blocks))
        # the free list is a ring; the next block to hand out is somewhere in it
        head_at = int(rng.integers(0, len(left)))
        s.update(tables=put(tables, torch.int32), lens=put(context, torch.int32),
                 new=put(new, torch.int32), ring=put(np.roll(left, head_at), torch.int32),
                 ring_state=put([head_at, len(left)], torch.int32), blocks=blocks,
                 capacity=int(max(1, new.sum())))
        s.update(lens_out=torch.empty_like(s["lens"]), ring_out=torch.empty_like(s["ring_state"]),
                 slots=torch.empty(s["capacity"], dtype=torch.int64, device=device),
                 positions=torch.empty(s["capacity"], dtype=torch.int32, device=device),
                 starts=torch.empty(len(new) + 1, dtype=torch.int32, device=device))
        if kind == "tables":
            return s
    dtype = TYPES[case["dtype"]]
    kv_heads, head = case["kv_heads"], case["head"]
    if kind in ("write", "gather"):
        tokens = case["tokens"]
        blocks = -(-tokens // block) + 3
        perm = rng.permutation(blocks)[:-(-tokens // block)]
        slots = (perm[:, None] * block + np.arange(block)).reshape(-1)[:tokens]
        s["slots"] = put(slots, torch.int64)
        s["key_out"] = torch.empty((tokens, kv_heads, head), dtype=dtype, device=device)
        s["value_out"] = torch.empty_like(s["key_out"])
        if kind == "gather":
            s["cache"] = _filled_cache(blocks, kv_heads, block, head, gen, device)
            return s
        s["cache"] = torch.zeros((blocks, kv_heads, block // 8, 9 * head), dtype=torch.uint8, device=device)
        # keys and values are slices of one projection's output, after its queries
        qkv = torch.cat([_normal((tokens, kv_heads * head), gen, device),
                         _outliers(_normal((tokens, kv_heads, head), gen, device)).flatten(1),
                         0.3 * _normal((tokens, kv_heads * head), gen, device)], dim=1).to(dtype)
        q, k, v = qkv.split(kv_heads * head, dim=1)
        s["key"], s["value"] = k.unflatten(1, (kv_heads, head)), v.unflatten(1, (kv_heads, head))
        return s
    heads = case["heads"]
    lens = _numbers(case["lens"], case["seed"])
    if kind == "decode":
        blocks = int((-(-lens // block)).sum()) + 3
        tables, _ = _tables(lens, block, 0, rng.permutation(blocks))
        s.update(tables=put(tables, torch.int32), lens=put(lens, torch.int32))
        s["query"] = (1.5 * _normal((len(lens), heads, head), gen, device)).to(dtype)
    else:
        tables = s["tables"].cpu().numpy()
        qkv = torch.cat([1.5 * _normal((len(lens), heads * head), gen, device),
                         _outliers(_normal((len(lens), kv_heads, head), gen, device)).flatten(1),
                         _normal((len(lens), kv_heads * head), gen, device)], dim=1).to(dtype)
        q, k, v = qkv.split([heads * head, kv_heads * head, kv_heads * head], dim=1)
        s["query"] = q.unflatten(1, (heads, head))
        s["key"], s["value"] = k.unflatten(1, (kv_heads, head)), v.unflatten(1, (kv_heads, head))
    s["cache"] = _filled_cache(blocks, kv_heads, block, head, gen, device)
    _kill_dead_rows(s["cache"], tables, lens, block, head)
    s["out"] = torch.empty((len(lens), heads, head), dtype=dtype, device=device)
    s["scale"] = head ** -0.5
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _quantise(x):
    """e2m1 codes, two to a byte, and e4m3 scales (as bytes) of groups of 16;
    a group with a NaN has a NaN scale."""
    g = x.float().unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    scale = (top / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    a = g.abs()
    # every border times a scale is exact in 32 bits; ties go to the even code
    code = ((a > 0.25 * s).to(torch.uint8) + (a >= 0.75 * s).to(torch.uint8) + (a > 1.25 * s).to(torch.uint8)
            + (a >= 1.75 * s).to(torch.uint8) + (a > 2.5 * s).to(torch.uint8) + (a >= 3.5 * s).to(torch.uint8)
            + (a > 5.0 * s).to(torch.uint8))
    code = torch.where(s > 0, code, torch.zeros_like(code))
    code = code + 8 * ((g < 0) & (code > 0)).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.view(torch.uint8)


def _values(codes, scales, tensor_scale):
    """The numbers that codes [..., D / 2] and scales [..., D / 16] stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=-1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() * tensor_scale
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _parts(tiles, head):
    """Key codes, value codes, key scales and value scales of tiles [..., 9 D], each [..., 8, n]."""
    g = head // 16
    kc = tiles[..., :4 * head].unflatten(-1, (8, head // 2))
    vc = tiles[..., 4 * head:8 * head].unflatten(-1, (g, 8, 8)).transpose(-3, -2).flatten(-2)
    ks = tiles[..., 8 * head:8 * head + 8 * g].unflatten(-1, (8, g))
    vs = tiles[..., 8 * head + 8 * g:].unflatten(-1, (g, 8)).transpose(-2, -1)
    return kc, vc, ks.contiguous(), vs.contiguous()


def _plain_gather(cache, slots, head, key_scale, value_scale, dtype):
    block = cache.shape[2] * 8
    tiles = cache[slots // block, :, slots % block // 8]
    n = torch.arange(slots.numel(), device=slots.device)
    kc, vc, ks, vs = (p[n, :, slots % 8].contiguous() for p in _parts(tiles, head))
    return _values(kc, ks, key_scale).to(dtype), _values(vc, vs, value_scale).to(dtype)


def _plain_write(cache, key, value, slots, head, key_scale, value_scale):
    kv_heads, tiles, size = cache.shape[1:]
    block, g = tiles * 8, head // 16
    device = cache.device
    kc, ks = _quantise(key.float() / key_scale)
    vc, vs = _quantise(value.float() / value_scale)
    base = ((slots // block * kv_heads)[:, None] + torch.arange(kv_heads, device=device)) * tiles
    base = ((base + (slots % block // 8)[:, None]) * size).unsqueeze(-1)
    row = (slots % 8)[:, None, None]
    group, eight = torch.arange(g, device=device), torch.arange(8, device=device)
    flat = cache.view(-1)
    flat[base + row * (head // 2) + torch.arange(head // 2, device=device)] = kc
    flat[base + 4 * head + row * 8 + (group[:, None] * 64 + eight).flatten()] = vc
    flat[base + 8 * head + row * g + group] = ks
    flat[base + 8 * head + 8 * g + row + group * 8] = vs


def _plain_decode(query, cache, tables, lens, scale, dtype):
    seqs, heads, head = query.shape
    kv_heads = cache.shape[1]
    longest = tables.shape[1] * cache.shape[2] * 8
    live = torch.arange(longest, device=lens.device) < lens[:, None]
    parts = _parts(cache[tables.long()].transpose(1, 2), head)  # [seqs, kv_heads, blocks, tiles, 8, n]
    kc, vc, ks, vs = (p.flatten(2, 4) for p in parts)
    mask = live[:, None, :, None]
    zero = torch.zeros((), device=lens.device)
    k = torch.where(mask, _values(kc, ks, 1.0), zero)
    v = torch.where(mask, _values(vc, vs, 1.0), zero)
    q = query.float().unflatten(1, (kv_heads, -1)) * scale
    x = torch.matmul(q, k.transpose(-2, -1))
    x = torch.where(live[:, None, None], x, torch.full_like(zero, -math.inf))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, zero, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(zero), total)
    return o.flatten(1, 2).to(dtype)


def _plain_tables(tables, lens, new, ring, state, block, capacity):
    lens, new = lens.long(), new.long()
    have = (lens + block - 1) // block
    need = (lens + new + block - 1) // block - have
    starts = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    first = need.cumsum(0) - need
    token = torch.arange(capacity, device=lens.device)
    live = token < starts[-1]
    r = torch.searchsorted(starts[1:], token, right=True).clamp(max=lens.numel() - 1)
    pos = torch.where(live, lens[r] + token - starts[r], torch.zeros_like(token))
    b = pos // block
    take = (state[0] + first[r] + b - have[r]) % ring.numel()
    ids = torch.where(live & (b >= have[r]), ring[take].long(), tables[r, b].long())
    opens = live & (b >= have[r])
    tables[r[opens], b[opens]] = ids[opens].int()
    none = torch.full_like(token, -1)
    used = need.sum()
    return {"tables": tables, "lens": (lens + new).int(),
            "ring": torch.stack([(state[0] + used) % ring.numel(), state[1] - used]).int(),
            "slots": torch.where(live, ids * block + pos % block, none),
            "positions": torch.where(live, pos, none).int(), "starts": starts.int()}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own_tables(s, pa):
    pa.pa_extend_tables(s["tables"], s["lens"], s["new"], s["block"], s["blocks"], s["slots"],
                        positions=s["positions"], token_starts=s["starts"],
                        seq_lens_out=s["lens_out"], free_blocks=s["ring"],
                        free_state=s["ring_state"], free_state_out=s["ring_out"])
    return {"tables": s["tables"], "lens": s["lens_out"], "ring": s["ring_out"],
            "slots": s["slots"], "positions": s["positions"], "starts": s["starts"]}


def _own_decode(s, pa, lens):
    if "workspace" not in s:  # allocated once, as a program does
        s["workspace"] = pa.alloc_workspace(
            pa.pa_decode_fp4_workspace_size(s["cache"], s["heads"]), s["cache"].device)
    pa.pa_decode_fp4(s["out"], s["query"], s["cache"], s["tables"], lens, s["scale"], s["workspace"])
    return s["out"]


def run(s):
    kind = s["kind"]
    if own:
        import paged_kv_cache_78_gb300 as pa
        if kind == "tables":
            return _own_tables(s, pa)
        if kind == "decode":
            return {"out": _own_decode(s, pa, s["lens"])}
        if kind == "step":
            t = _own_tables(s, pa)
            pa.pa_reshape_and_cache_fp4(s["cache"], s["key"], s["value"], s["slots"])
            return dict(t, out=_own_decode(s, pa, s["lens_out"]))
        scales = {"key_scale": s["key_scale"], "value_scale": s["value_scale"]}
        if kind == "write":
            pa.pa_reshape_and_cache_fp4(s["cache"], s["key"], s["value"], s["slots"], **scales)
        pa.pa_gather_cache_fp4(s["key_out"], s["value_out"], s["cache"], s["slots"], **scales)
        return {"key": s["key_out"], "value": s["value_out"]}
    if kind == "tables":
        return _plain_tables(s["tables"], s["lens"], s["new"], s["ring"], s["ring_state"],
                             s["block"], s["capacity"])
    dtype = TYPES[s["dtype"]]
    if kind == "decode":
        return {"out": _plain_decode(s["query"], s["cache"], s["tables"], s["lens"], s["scale"], dtype)}
    if kind == "step":
        t = _plain_tables(s["tables"], s["lens"], s["new"], s["ring"], s["ring_state"], s["block"],
                          s["capacity"])
        _plain_write(s["cache"], s["key"], s["value"], t["slots"], s["head"], 1.0, 1.0)
        return dict(t, out=_plain_decode(s["query"], s["cache"], t["tables"], t["lens"], s["scale"], dtype))
    scales = (s["key_scale"], s["value_scale"])
    if kind == "write":
        _plain_write(s["cache"], s["key"], s["value"], s["slots"], s["head"], *scales)
    k, v = _plain_gather(s["cache"], s["slots"], s["head"], *scales, dtype)
    return {"key": k, "value": v}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def _exact_table():
    """The 127 non-negative e4m3 numbers by their codes (a bit of sign, four
    of exponent with bias 7, three of mantissa), and the eight of e2m1."""
    e4m3 = [m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            for e in range(16) for m in range(8)][:127]
    return (torch.tensor(e4m3, dtype=torch.float64, device="cuda"),
            torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda"))


def _exact_nearest(table, x):
    """The nearest entry of an ascending table, ties to its even places."""
    hi = torch.searchsorted(table, x.contiguous()).clamp(1, len(table) - 1)
    below, above = x - table[hi - 1], table[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return table[torch.where(up, hi, hi - 1)]


def _exact_rounded(x, tensor_scale):
    """What [..., D] becomes in the cache."""
    e4m3, e2m1 = _exact_table()
    x = x.double().unflatten(-1, (-1, 16)) / tensor_scale
    s = _exact_nearest(e4m3, x.abs().amax(-1, keepdim=True) / 6)
    code = _exact_nearest(e2m1, torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0))
    return (torch.sign(x) * code * s * tensor_scale).flatten(-2)


def _exact_read(cache, slots, head, tensor_scale, values):
    """Keys or values [n, kv_heads, D] of slots, each element fetched by its own byte's address."""
    e4m3, e2m1 = _exact_table()
    kv_heads, tiles, size = cache.shape[1:]
    d = torch.arange(head, device=cache.device)
    h = torch.arange(kv_heads, device=cache.device)[:, None]
    slot = slots[:, None, None]
    tile = ((slot // (8 * tiles)) * kv_heads + h) * tiles + slot % (8 * tiles) // 8
    row = slot % 8
    if values:
        code_at = 4 * head + (d // 16) * 64 + row * 8 + d % 16 // 2
        scale_at = 8 * head + head // 2 + (d // 16) * 8 + row
    else:
        code_at = row * (head // 2) + d // 2
        scale_at = 8 * head + row * (head // 16) + d // 16
    flat = cache.view(-1)
    nibble = (flat[tile * size + code_at].long() >> (4 * (d % 2))) & 15
    v = e2m1[nibble & 7] * (1 - 2 * (nibble >> 3)).double()
    return v * e4m3[flat[tile * size + scale_at].long() & 127] * tensor_scale


def exact(case, seed):
    kind = case["kind"]
    if kind == "tables":
        return None  # whole numbers, which are compared as they are
    s = prepare(case, seed)
    if kind == "write":
        return {"key": _exact_rounded(s["key"], case["key_scale"]),
                "value": _exact_rounded(s["value"], case["value_scale"])}
    if kind == "gather":
        return {n: torch.cat([_exact_read(s["cache"], p, case["head"], case[n + "_scale"], n == "value")
                              for p in s["slots"].split(8192)]) for n in ("key", "value")}
    head, block, group = case["head"], case["block"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if kind == "step":
        new_k, new_v = _exact_rounded(s["key"], 1.0), _exact_rounded(s["value"], 1.0)
    for r, n in enumerate(s["lens"].tolist()):
        pos = torch.arange(n, device="cuda")
        slots = s["tables"][r].long()[pos // block] * block + pos % block
        k = _exact_read(s["cache"], slots, head, 1.0, False)
        v = _exact_read(s["cache"], slots, head, 1.0, True)
        if kind == "step":
            k, v = torch.cat([k, new_k[r:r + 1]]), torch.cat([v, new_v[r:r + 1]])
        if k.shape[0]:
            q = s["query"][r].double().unflatten(0, (-1, group))
            w = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * float(s["scale"]), dim=-1)
            out[r] = torch.einsum("hgn,nhd->hgd", w, v).flatten(0, 1)
    if kind == "decode":
        return {"out": out}
    return {"tables": None, "lens": None, "ring": None, "slots": None, "positions": None,
            "starts": None, "out": out}
