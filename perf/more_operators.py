"""The 8-bit paged cache's operators and the two around them, as measured work: the
same calls in their plain form (elementary torch operations, 32 bits or more) and,
where `own` is true, through this repository's entry points.

An 8-bit cache is an int8 tensor [num_blocks, num_kv_heads, block_size / 8,
16 * (head_size + 1)]; the last axis is a tile of eight tokens, as bytes:
    fp32, fp32, 8 zeros               key scale and value scale of the tile's block and head
    [head_size / 16][8 tokens][16]    key codes plus 128
    [head_size / 16][8 tokens][16]    value codes plus 128
A number is code * scale, with one scale for a block's keys of a head and one for its
values (each tile of the block repeats them).  A write that begins a block sets its
scale to max|x| / 127 over the tokens that it puts there; a write behind other tokens
raises the scale where it has to, and rounds the codes that are there again.

Kinds of cases: "rope" (norms of queries and keys for each head, and the rotation by
position), "write" (new tokens into the cache, and the touched blocks read back),
"gather" (cached tokens read back), "decode" (one query token per sequence; with
`weights` also the attention that each block got, added up over the steps), "evict"
(the blocks with the least of it leave their sequences) and "step" (a decode step
with all of them in a row).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LARGEST_BYTES = 500_000_000  # of a drawn case, about: the largest listed one's are 538 million
DECAY = 0.96875


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode batch's queries and keys, slices of the projection's output
        {"name": "rope_decode", "kind": "rope", "tokens": 64, "heads": 14, "kv_heads": 2, "head": 64,
         "rotary": 64, "interleaved": False, "dtype": "bf16", "far": 32768, "offsets": True},
        # a prompt chunk, far into long sequences
        {"name": "rope_prefill", "kind": "rope", "tokens": 16381, "heads": 32, "kv_heads": 8,
         "head": 128, "rotary": 128, "interleaved": False, "dtype": "bf16", "far": 131072,
         "offsets": False},
        # the newest tokens of a decode batch, behind others in their blocks
        {"name": "write_decode", "kind": "write", "requests": 64, "new": 1, "kv_heads": 2, "head": 64,
         "block": 16, "dtype": "bf16", "seed": 21},
        # prompt chunks of several requests, each of which continues a block
        {"name": "write_prefill", "kind": "write", "requests": 5, "new": 3277, "kv_heads": 8,
         "head": 128, "block": 16, "dtype": "bf16", "seed": 22},
        # a long cached context read back for a prompt chunk's attention
        {"name": "gather_context", "kind": "gather", "tokens": 65536, "kv_heads": 8, "head": 128,
         "block": 16, "dtype": "bf16"},
        # the smallest batch: a few short sequences, latency
        {"name": "decode_tiny", "kind": "decode", "lens": "list:7,16,33,100", "heads": 4,
         "kv_heads": 4, "head": 64, "block": 8, "dtype": "bf16", "weights": False, "seed": 41},
        # grouped queries, ragged lengths, the blocks' weights kept for eviction
        {"name": "decode_gqa", "kind": "decode", "lens": "uniform:0:2048*64", "heads": 14,
         "kv_heads": 2, "head": 64, "block": 16, "dtype": "bf16", "weights": True, "seed": 42},
        # long contexts, the bound on memory
        {"name": "decode_long", "kind": "decode", "lens": "fixed:32768*8", "heads": 32,
         "kv_heads": 8, "head": 128, "block": 16, "dtype": "bf16", "weights": False, "seed": 44},
        # very different lengths (one sequence still empty), wide heads, 32-bit queries
        {"name": "decode_mixed_fp32", "kind": "decode", "lens": "list:0,1,513,4097,40001",
         "heads": 16, "kv_heads": 2, "head": 256, "block": 16, "dtype": "fp32", "weights": True,
         "seed": 45},
        # a serving step: sequences about as long as they may be, a block or two too many
        {"name": "evict_step", "kind": "evict", "lens": "uniform:1000:2080*256", "block": 16,
         "budget": 128, "first": 1, "last": 4, "seed": 61},
        # long prompts cut to a quarter at once
        {"name": "evict_prompt", "kind": "evict", "lens": "uniform:100000:131072*16", "block": 16,
         "budget": 2048, "first": 4, "last": 64, "seed": 62},
        # a whole decode step: eviction, tables, norms and rotation, write, attention
        {"name": "step_gqa", "kind": "step", "lens": "uniform:0:2100*128", "heads": 32,
         "kv_heads": 8, "head": 128, "block": 16, "dtype": "bf16", "budget": 128, "first": 1,
         "last": 4, "far": 32768, "seed": 51},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("rope", "write", "gather", "decode", "decode", "decode", "evict", "step"))
    seed = rng.randrange(1 << 30)
    block = rng.choice((8, 16, 16, 32, 64, 128, 256))
    if kind == "evict":
        seqs = _log_int(rng, 1, 1000)
        longest = _log_int(rng, block, min(131072 * block // 16, max(block, 2_000_000 // seqs * block)))
        blocks = -(-longest // block)
        first, last = rng.choice((0, 1, 4)), rng.choice((1, 2, 32))
        return {"kind": kind, "lens": "uniform:%d:%d*%d" % (longest // 3, longest, seqs), "block": block,
                "budget": max(first + last, _log_int(rng, 1, blocks)), "first": first, "last": last,
                "seed": seed}
    head = rng.choice((64, 128, 128, 256))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    elem = 2 if dtype == "bf16" else 4
    kv_heads = rng.choice((1, 2, 4, 5, 8))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 8, 12, 16))
    if kind == "rope":
        most = max(2, int(LARGEST_BYTES / (2.5 * elem * kv_heads * (group + 1) * head)))
        return {"kind": kind, "tokens": _log_int(rng, 1, min(65536, most)), "heads": kv_heads * group,
                "kv_heads": kv_heads, "head": head, "rotary": rng.choice((head, head, head // 2, 32)),
                "interleaved": rng.random() < 0.3, "dtype": dtype, "far": _log_int(rng, 256, 131072),
                "offsets": rng.random() < 0.5}
    if kind in ("write", "gather"):
        kv_heads = rng.choice((1, 2, 3, 4, 8, 16, 40))
        most = max(2, min(65536, int(LARGEST_BYTES / (kv_heads * head * (2 * elem + 2))) //
                          (1 if kind == "gather" else 2)))
        tokens = _log_int(rng, 1, most)
        if kind == "gather":
            return {"kind": kind, "tokens": tokens, "kv_heads": kv_heads, "head": head, "block": block,
                    "dtype": dtype}
        # a request may have its whole first block read back
        requests = _log_int(rng, 1, max(1, min(1024, most // (2 * block))))
        new = 1 if rng.random() < 0.5 else max(1, tokens // requests - block)
        return {"kind": kind, "requests": requests, "new": new, "kv_heads": kv_heads, "head": head,
                "block": block, "dtype": dtype, "seed": seed}
    seqs = _log_int(rng, 1, 256)
    most = max(1, min(131072, LARGEST_BYTES // 2 // (seqs * kv_heads * head * 2)))
    longest = _log_int(rng, 1, most)
    case = {"kind": kind, "lens": rng.choice(("uniform:%d:%d*%d" % (rng.choice((0, 1)), longest, seqs),
                                              "fixed:%d*%d" % (longest, seqs))),
            "heads": kv_heads * group, "kv_heads": kv_heads, "head": head, "block": block, "dtype": dtype,
            "seed": seed}
    if kind == "decode":
        return dict(case, weights=rng.random() < 0.5)
    blocks = -(-longest // block)
    return dict(case, budget=max(3, _log_int(rng, 1, blocks)), first=1, last=2,
                far=longest + 100 * block + 1)


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


def _evicted(case, lens):
    """Blocks that leave each sequence."""
    return np.maximum(-(-lens // case["block"]) - case["budget"], 0)


def _rope_work(tokens, heads, head, rotary, elem):
    # rows in and out, positions, a row of the table for each token, the norms' weights
    return {"bytes": tokens * (2 * heads * head * elem + 4 + 4 * rotary) + 2 * head * elem,
            "flops": tokens * heads * (4 * head + 3 * rotary)}


def work(case):
    kind = case["kind"]
    if kind == "evict":
        lens = _numbers(case["lens"], case["seed"])
        n, out = -(-lens // case["block"]), _evicted(case, lens)
        cut = n[out > 0]
        # tables and weights of every sequence in and out; lengths and counts; the ring
        return {"bytes": int(16 * n.sum() + 4 * out.sum()) + 16 * len(lens) + 16, "flops": int(cut.sum())}
    elem = 2 if case["dtype"] == "bf16" else 4
    if kind == "rope":
        w = _rope_work(case["tokens"], case["heads"] + case["kv_heads"], case["head"], case["rotary"], elem)
        w["bytes"] += 4 * case["tokens"] * case["offsets"]
        return w
    kv_heads, head, block = case["kv_heads"], case["head"], case["block"]
    row = 2 * kv_heads * head
    if kind == "gather":
        n = case["tokens"]
        return {"bytes": n * (row * (elem + 1) + 8) + -(-n // block) * 8 * kv_heads, "flops": 0}
    if kind == "write":
        new, n = case["new"], case["requests"] * case["new"]
        back = case["requests"] * (new + block // 2)  # half a block is there already
        blocks = case["requests"] * (-(-new // block) + 1)
        return {"bytes": n * (row * (elem + 1) + 8) + back * (row * (elem + 1) + 8)
                + 16 * kv_heads * blocks, "flops": 0}
    lens, bytes_, flops = _numbers(case["lens"], case["seed"]), 0, 0
    heads, seqs = case["heads"], len(lens)
    weights = kind == "step" or case["weights"]
    if kind == "step":
        out = _evicted(case, lens)
        n = -(-lens // block)
        lens = lens - out * block + 1
        r = _rope_work(seqs, heads + kv_heads, head, head, elem)
        # eviction, tables, norms and rotation, the write
        bytes_ = int(16 * n.sum()) + 32 * seqs + r["bytes"] + seqs * (row * (elem + 1) + 24 + 16 * kv_heads)
        flops = r["flops"]
    tokens, blocks = int(lens.sum()), int((-(-lens // block)).sum())
    bytes_ += tokens * row + blocks * (8 * kv_heads + 4 + 8 * weights) + 4 * seqs
    return {"bytes": bytes_ + 2 * seqs * heads * head * elem, "flops": flops + 4 * tokens * heads * head}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(shape, gen, device):
    return torch.randn(shape, generator=gen, device=device, dtype=torch.float32)


def _outliers(x):
    """A few channels an order larger than the others, as keys have them."""
    x[..., 3::37] *= 6.0
    return x


def _codes(x, scale):
    """Codes plus 128 of x [..., block, D] with scales [...]: the nearest, ties to even."""
    s = scale.double()[..., None, None]
    q = torch.where(s > 0, x.double() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))
    return (q.round().clamp(-127, 127) + 128).to(torch.uint8)


def _pack(kc, vc, ks, vs):
    """Blocks [..., block / 8, 16 (D + 1)] of codes [..., block, D] and scales [...]."""
    tiles = kc.shape[-2] // 8
    head = torch.zeros(ks.shape + (tiles, 4), dtype=torch.float32, device=ks.device)
    head[..., 0], head[..., 1] = ks[..., None], vs[..., None]
    parts = [c.unflatten(-2, (tiles, 8)).unflatten(-1, (-1, 16)).transpose(-3, -2).flatten(-3)
             for c in (kc, vc)]
    return torch.cat([head.view(torch.uint8)] + parts, dim=-1).view(torch.int8)


def _filled_cache(blocks, kv_heads, block, head, gen, device):
    """A pool of quantised normal keys and values, each block with scales of its own."""
    cache = torch.empty((blocks, kv_heads, block // 8, 16 * (head + 1)), dtype=torch.int8, device=device)
    step = max(1, (1 << 23) // (kv_heads * block * head))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        k = _outliers(_normal((n, kv_heads, block, head), gen, device))
        v = _normal((n, kv_heads, block, head), gen, device)
        ks, vs = ((x.abs().amax((-2, -1)) / 127.0) for x in (k, v))
        cache[b:b + n] = _pack(_codes(k, ks), _codes(v, vs), ks, vs)
    return cache


def _tables(lens, block, extra, perm):
    """Block tables that take `perm` in order, and the ids that are left."""
    counts = -(-lens // block)
    tables = np.zeros((len(lens), int(max(1, (-(-(lens + extra) // block)).max()))), dtype=np.int32)
    at = 0
    for r, c in enumerate(counts):
        tables[r, :c] = perm[at:at + c]
        at += int(c)
    return tables, perm[at:]


def _cos_sin(far, rotary, device):
    """[position][rotary]: cosines, then sines, of position / 10000^(2 i / rotary)."""
    rate = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64, device=device) * 2 / rotary)
    a = torch.arange(far, dtype=torch.float64, device=device)[:, None] * rate
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    kind = case["kind"]

    def put(a, dtype):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(device)

    s = dict(case)
    if kind in ("evict", "step"):
        lens = _numbers(case["lens"], case["seed"])
        extra, block = int(kind == "step"), case["block"]
        blocks = int((-(-(lens + extra) // block)).sum()) + 7
        tables, left = _tables(lens, block, extra, rng.permutation(blocks))
        # the free blocks are a ring with room for all; its front is somewhere in it
        ring, front = np.zeros(blocks, dtype=np.int64), int(rng.integers(0, blocks))
        ring[(front + np.arange(len(left))) % blocks] = left
        # weights as attention leaves them: few blocks with most, many with next to nothing
        weights = np.exp(1.5 * rng.standard_normal(tables.shape)).astype(np.float32)
        weights[np.arange(tables.shape[1]) >= (-(-lens // block))[:, None]] = 0
        s.update(tables=put(tables, torch.int32), lens=put(lens, torch.int32), ring=put(ring, torch.int32),
                 ring_state=put([front, len(left)], torch.int32), weights=put(weights, torch.float32),
                 gone=put(rng.integers(0, 100, len(lens)) * block, torch.int32), blocks=blocks)
        for n in ("tables", "lens", "ring_state", "weights", "gone"):  # the state after the call
            s[n + "_out"] = s[n].clone()
        if kind == "evict":
            return s
    dtype = TYPES[case["dtype"]]
    if kind == "rope":
        n, heads, kv_heads, head = (case[x] for x in ("tokens", "heads", "kv_heads", "head"))
        # queries and keys are slices of one projection's output, with the values behind
        qkv = _outliers(_normal((n, heads + 2 * kv_heads, head), gen, device)).flatten(1).to(dtype)
        q, k = qkv[:, :heads * head], qkv[:, heads * head:(heads + kv_heads) * head]
        s.update(query=q.unflatten(1, (heads, head)), key=k.unflatten(1, (kv_heads, head)),
                 positions=put(rng.integers(0, case["far"] // 2, n), torch.int32),
                 shift=put(rng.integers(0, case["far"] // 2, n), torch.int32) if case["offsets"] else None)
        s.update(query_out=torch.empty((n, heads, head), dtype=dtype, device=device),
                 key_out=torch.empty((n, kv_heads, head), dtype=dtype, device=device))
    if kind in ("rope", "step"):
        s["cos_sin"] = _cos_sin(case["far"], case.get("rotary", case["head"]), device)
        for n in ("query_weight", "key_weight"):
            s[n] = (1.0 + 0.2 * _normal((case["head"],), gen, device)).to(dtype)
        s["eps"] = 1e-6
        if kind == "rope":
            return s
    kv_heads, head, block = case["kv_heads"], case["head"], case["block"]
    if kind in ("write", "gather"):
        if kind == "gather":
            have, new = np.zeros(1, dtype=np.int64), np.array([case["tokens"]])
        else:  # what each request's first block holds already, and its new tokens
            have = np.random.default_rng(case["seed"]).integers(0, block, case["requests"])
            new = np.full(case["requests"], case["new"])
        blocks = int((-(-(have + new) // block)).sum()) + 3
        tables, _ = _tables(have + new, block, 0, rng.permutation(blocks))
        every = [t[np.arange(n) // block].astype(np.int64) * block + np.arange(n) % block
                 for t, n in zip(tables, have + new)]
        s["slots"] = put(np.concatenate([e[h:] for e, h in zip(every, have)]), torch.int64)
        s["back"] = put(np.concatenate(every), torch.int64)
        s["cache"] = _filled_cache(blocks, kv_heads, block, head, gen, device)
        s["key_out"] = torch.empty((len(s["back"]), kv_heads, head), dtype=dtype, device=device)
        s["value_out"] = torch.empty_like(s["key_out"])
        if kind == "gather":
            return s
        # keys and values are slices of one projection's output, after its queries
        n = len(s["slots"])
        qkv = torch.cat([_normal((n, kv_heads * head), gen, device),
                         _outliers(_normal((n, kv_heads, head), gen, device)).flatten(1),
                         _normal((n, kv_heads * head), gen, device)], dim=1).to(dtype)
        _, k, v = qkv.split(kv_heads * head, dim=1)
        s["key"], s["value"] = k.unflatten(1, (kv_heads, head)), v.unflatten(1, (kv_heads, head))
        return s
    heads = case["heads"]
    if kind == "decode":
        lens = _numbers(case["lens"], case["seed"])
        blocks = int((-(-lens // block)).sum()) + 3
        tables, _ = _tables(lens, block, 0, rng.permutation(blocks))
        s.update(tables=put(tables, torch.int32), lens=put(lens, torch.int32))
        s["query"] = (1.5 * _normal((len(lens), heads, head), gen, device)).to(dtype)
        if case["weights"]:
            old = np.exp(rng.standard_normal(tables.shape))
            old[np.arange(tables.shape[1]) >= (-(-lens // block))[:, None]] = 0
            s["weights"] = put(old, torch.float32)
            s["weights_out"] = torch.zeros_like(s["weights"])
    else:
        qkv = torch.cat([_outliers(_normal((len(lens), heads + kv_heads, head), gen, device)).flatten(1),
                         _normal((len(lens), kv_heads * head), gen, device)], dim=1).to(dtype)
        q, k, v = qkv.split([heads * head, kv_heads * head, kv_heads * head], dim=1)
        s["raw_query"] = q.unflatten(1, (heads, head))
        s["raw_key"], s["value"] = k.unflatten(1, (kv_heads, head)), v.unflatten(1, (kv_heads, head))
        s["query"] = torch.empty((len(lens), heads, head), dtype=dtype, device=device)
        s["key"] = torch.empty((len(lens), kv_heads, head), dtype=dtype, device=device)
        s["one"] = torch.ones_like(s["lens"])
        s["slots"] = torch.empty(len(lens), dtype=torch.int64, device=device)
        s["positions"] = torch.empty(len(lens), dtype=torch.int32, device=device)
        s["next_lens"], s["next_ring"] = torch.empty_like(s["lens"]), torch.empty_like(s["ring_state"])
        s["next_weights"] = torch.zeros_like(s["weights"])
        s["start_tables"] = s["tables"]
    s["cache"] = _filled_cache(blocks, kv_heads, block, head, gen, device)
    s["out"] = torch.empty((len(lens), heads, head), dtype=dtype, device=device)
    s["scale"] = head ** -0.5
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _plain_rope(x, weight, cos_sin, at, interleaved, eps):
    f = x.float()
    f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + eps) * weight.float()
    rotary = cos_sin.shape[1]
    c, sn = cos_sin[at.long()].unsqueeze(1).split(rotary // 2, dim=-1)
    turn, rest = f[..., :rotary], f[..., rotary:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * c - b * sn, b * c + a * sn], dim=-1).flatten(-2)
    else:
        a, b = turn.chunk(2, dim=-1)
        turn = torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)
    return torch.cat([turn, rest], dim=-1).to(x.dtype)


def _parts(tiles, head):
    """Key and value codes [..., 8, D] (no longer plus 128) and scales [...] of tiles."""
    b = tiles.view(torch.uint8)
    scales = b[..., :8].contiguous().view(torch.float32)
    codes = [b[..., at:at + 8 * head].unflatten(-1, (head // 16, 8, 16)).transpose(-3, -2).flatten(-2)
             .to(torch.int16) - 128 for at in (16, 16 + 8 * head)]
    return codes[0], codes[1], scales[..., 0], scales[..., 1]


def _blocks(tiles, head):
    """The same of whole blocks [..., block / 8, 16 (D + 1)]: codes [..., block, D]."""
    kc, vc, ks, vs = _parts(tiles, head)
    return kc.flatten(-3, -2), vc.flatten(-3, -2), ks[..., 0], vs[..., 0]


def _plain_gather(cache, slots, head, dtype):
    block = cache.shape[2] * 8
    out = []
    for part in slots.split(16384):
        tiles = cache[part // block, :, part % block // 8]
        n = torch.arange(part.numel(), device=slots.device)
        kc, vc, ks, vs = _parts(tiles, head)
        out.append([(c[n, :, part % 8].float() * sc[..., None]).to(dtype) for c, sc in ((kc, ks), (vc, vs))])
    return torch.cat([o[0] for o in out]), torch.cat([o[1] for o in out])


def _plain_write(cache, key, value, slots, head):
    """Block by block: the blocks that get tokens, what they hold, their new scales."""
    kv_heads, block = cache.shape[1], cache.shape[2] * 8
    ids, at = torch.unique(slots // block, return_inverse=True)
    step = max(1, (1 << 26) // (kv_heads * block * head))
    for i0 in range(0, ids.numel(), step):
        part = ids[i0:i0 + step]
        mine = (at >= i0) & (at < i0 + step)
        i, off = at[mine] - i0, slots[mine] % block
        new = torch.zeros((part.numel(), block), dtype=torch.bool, device=slots.device)
        new[i, off] = True
        begins = new[:, 0]
        kc, vc, ks, vs = _blocks(cache[part], head)
        after = []
        for codes, scale, x in ((kc, ks, key), (vc, vs, value)):
            rows = torch.zeros((part.numel(), block, kv_heads, head), dtype=torch.float32, device=slots.device)
            rows[i, off] = x[mine].float()
            rows = rows.transpose(1, 2)
            old = torch.where(begins[:, None], torch.zeros_like(scale), scale)
            s = torch.maximum(old, (rows.abs().amax((-2, -1)).double() / 127.0).float())
            held = codes.double() * scale.double()[..., None, None]  # exact
            x = torch.where(new[:, None, :, None], rows.double(), held)
            moved = new[:, None, :, None] | ((s > old) & ~begins[:, None])[..., None, None]
            c = torch.where(moved, _codes(x, s), (codes + 128).to(torch.uint8))
            after += [c, s]
        cache[part] = _pack(after[0], after[2], after[1], after[3])


def _plain_decode(query, cache, tables, lens, scale, dtype, old=None):
    seqs, heads, head = query.shape
    kv_heads, block = cache.shape[1], cache.shape[2] * 8
    live = torch.arange(tables.shape[1] * block, device=lens.device) < lens[:, None]
    kc, vc, ks, vs = _blocks(cache[tables.long()].transpose(1, 2), head)  # [seqs, kv_heads, blocks, block, D]
    k = (kc.float() * ks[..., None, None]).flatten(2, 3)
    q = query.float().unflatten(1, (kv_heads, -1)) * scale
    x = torch.matmul(q, k.transpose(-2, -1))
    del kc, k
    zero = torch.zeros((), device=lens.device)
    x = torch.where(live[:, None, None], x, torch.full_like(zero, -math.inf))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, zero, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(zero), total)
    v = torch.where(live[:, None, :, None], (vc.float() * vs[..., None, None]).flatten(2, 3), zero)
    o = torch.matmul(p, v).flatten(1, 2).to(dtype)
    if old is None:
        return o
    w = p.sum((1, 2)).unflatten(1, (-1, block)).sum(-1)
    has = torch.arange(tables.shape[1], device=lens.device) * block < lens[:, None]
    return o, torch.where(has, DECAY * old + w, torch.zeros_like(w))


def _plain_evict(tables, weights, lens, gone, ring, state, case):
    block, budget, first, last = (case[x] for x in ("block", "budget", "first", "last"))
    col = torch.arange(tables.shape[1], device=lens.device)
    n = ((lens.long() + block - 1) // block)[:, None]
    out = (n - budget).clamp(min=0)
    may = (col >= first) & (col < n - last)
    order = torch.sort(torch.where(may, weights, torch.full_like(weights, math.inf)), dim=1, stable=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, col.expand_as(order).contiguous())
    leaves = (rank < out) & may
    stays = ~leaves & (col < n)
    to = torch.where(stays, stays.cumsum(1) - 1,
                     torch.where(leaves, n - out + leaves.cumsum(1) - 1, col.expand_as(order)))
    new_tables = torch.empty_like(tables).scatter_(1, to, tables)
    new_weights = torch.empty_like(weights).scatter_(
        1, to, torch.where(leaves, torch.zeros_like(weights), weights))
    total = out.sum()
    at = torch.where(leaves, (state[0] + state[1] + leaves.flatten().cumsum(0).view_as(leaves) - 1) % ring.numel(), -1)
    ring[at[leaves]] = tables[leaves]
    moved = (out[:, 0] * block).int()
    return {"tables": new_tables, "weights": new_weights, "lens": lens - moved, "gone": gone + moved,
            "ring": ring, "ring_state": torch.stack([state[0], state[1] + total]).int()}


def _plain_extend(tables, lens, ring, state, block):
    """One token more for every sequence."""
    tables, b = tables.clone(), lens.long() // block
    opens = lens % block == 0
    take = (state[0] + opens.cumsum(0) - 1) % ring.numel()
    r = torch.arange(lens.numel(), device=lens.device)
    ids = torch.where(opens, ring[take], tables[r, b])
    tables[r, b] = ids
    used = opens.sum()
    return (tables, (lens + 1).int(), torch.stack([(state[0] + used) % ring.numel(), state[1] - used]).int(),
            ids.long() * block + lens % block, lens)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _workspace(s, pa, tables, weights):
    if "workspace" not in s:  # allocated once, as a program does
        s["workspace"] = pa.alloc_workspace(
            pa.pa_decode_int8_workspace_size(s["cache"], s["heads"], tables if weights else None),
            s["cache"].device)
    return s["workspace"]


def _own_evict(s, pa):
    pa.pa_evict_blocks(s["tables"], s["weights"], s["lens"], s["block"], s["budget"], s["first"], s["last"],
                       free_blocks=s["ring"], free_state=s["ring_state"], evicted_tokens=s["gone"],
                       block_tables_out=s["tables_out"], block_weights_out=s["weights_out"],
                       seq_lens_out=s["lens_out"], free_state_out=s["ring_state_out"],
                       evicted_tokens_out=s["gone_out"])
    return {"tables": s["tables_out"], "weights": s["weights_out"], "lens": s["lens_out"],
            "gone": s["gone_out"], "ring": s["ring"], "ring_state": s["ring_state_out"]}


def _own(s, pa):
    kind = s["kind"]
    if kind == "rope":
        pa.pa_norm_rope(s["query_out"], s["key_out"], s["query"], s["key"], s["query_weight"],
                        s["key_weight"], s["cos_sin"], s["positions"], s["eps"], s["interleaved"],
                        position_offsets=s["shift"])
        return {"query": s["query_out"], "key": s["key_out"]}
    if kind == "evict":
        return _own_evict(s, pa)
    if kind in ("write", "gather"):
        if kind == "write":
            pa.pa_reshape_and_cache_int8(s["cache"], s["key"], s["value"], s["slots"])
        pa.pa_gather_cache_int8(s["key_out"], s["value_out"], s["cache"], s["back"])
        return {"key": s["key_out"], "value": s["value_out"]}
    if kind == "decode":
        keep = {}
        if s["weights"] is not False:
            keep = {"block_weights": s["weights"], "block_weights_out": s["weights_out"], "decay": DECAY}
        pa.pa_decode_int8(s["out"], s["query"], s["cache"], s["tables"], s["lens"], s["scale"],
                          _workspace(s, pa, s["tables"], bool(keep)), **keep)
        return {"out": s["out"], "weights": s["weights_out"]} if keep else {"out": s["out"]}
    e = _own_evict(s, pa)
    pa.pa_extend_tables(e["tables"], e["lens"], s["one"], s["block"], s["blocks"], s["slots"],
                        positions=s["positions"], seq_lens_out=s["next_lens"], free_blocks=e["ring"],
                        free_state=e["ring_state"], free_state_out=s["next_ring"])
    pa.pa_norm_rope(s["query"], s["key"], s["raw_query"], s["raw_key"], s["query_weight"], s["key_weight"],
                    s["cos_sin"], s["positions"], s["eps"], position_offsets=e["gone"])
    pa.pa_reshape_and_cache_int8(s["cache"], s["key"], s["value"], s["slots"])
    pa.pa_decode_int8(s["out"], s["query"], s["cache"], e["tables"], s["next_lens"], s["scale"],
                      _workspace(s, pa, e["tables"], True), block_weights=e["weights"],
                      block_weights_out=s["next_weights"], decay=DECAY)
    return {"tables": e["tables"], "lens": s["next_lens"], "ring_state": s["next_ring"], "gone": e["gone"],
            "query": s["query"], "out": s["out"], "weights": s["next_weights"]}


def run(s):
    if own:
        import paged_kv_cache_78_gb300 as pa
        return _own(s, pa)
    kind = s["kind"]
    if kind == "evict":
        return _plain_evict(s["tables"], s["weights"], s["lens"], s["gone"], s["ring"], s["ring_state"], s)
    dtype = TYPES[s["dtype"]]
    if kind == "rope":
        at = s["positions"] if s["shift"] is None else s["positions"] + s["shift"]
        return {n: _plain_rope(s[n], s[n + "_weight"], s["cos_sin"], at, s["interleaved"], s["eps"])
                for n in ("query", "key")}
    if kind in ("write", "gather"):
        if kind == "write":
            _plain_write(s["cache"], s["key"], s["value"], s["slots"], s["head"])
        k, v = _plain_gather(s["cache"], s["back"], s["head"], dtype)
        return {"key": k, "value": v}
    if kind == "decode":
        old = s["weights"] if s["weights"] is not False else None
        o = _plain_decode(s["query"], s["cache"], s["tables"], s["lens"], s["scale"], dtype, old)
        return {"out": o} if old is None else {"out": o[0], "weights": o[1]}
    e = _plain_evict(s["tables"], s["weights"], s["lens"], s["gone"], s["ring"], s["ring_state"], s)
    tables, lens, state, slots, at = _plain_extend(e["tables"], e["lens"], e["ring"], e["ring_state"], s["block"])
    at = at + e["gone"]
    q = _plain_rope(s["raw_query"], s["query_weight"], s["cos_sin"], at, False, s["eps"])
    k = _plain_rope(s["raw_key"], s["key_weight"], s["cos_sin"], at, False, s["eps"])
    _plain_write(s["cache"], k, s["value"], slots, s["head"])
    o, w = _plain_decode(q, s["cache"], tables, lens, s["scale"], dtype, e["weights"])
    return {"tables": tables, "lens": lens, "ring_state": state, "gone": e["gone"], "query": q, "out": o,
            "weights": w}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def _exact_rope(x, weight, cos_sin, at, interleaved, eps):
    d, rotary = x.shape[-1], cos_sin.shape[1]
    x = x.double()
    x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + eps) * weight.double()
    i = torch.arange(rotary // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    turn = cos_sin[at.long()].double()[:, None, :]
    turn = torch.complex(turn[..., :rotary // 2], turn[..., rotary // 2:])
    z = torch.complex(x[..., a], x[..., b]) * turn
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_read(cache, slots, head):
    """Keys and values [n, kv_heads, D], each element fetched by its own byte's address."""
    kv_heads, tiles, size = cache.shape[1:]
    flat = cache.view(torch.uint8).view(-1)
    scales = cache.view(torch.uint8).view(-1).view(torch.float32)
    d = torch.arange(head, device=cache.device)
    tile = (slots // (8 * tiles))[:, None] * kv_heads + torch.arange(kv_heads, device=cache.device)
    base = ((tile * tiles + (slots % (8 * tiles) // 8)[:, None]) * size)[..., None]
    at = base + 16 + d // 16 * 128 + (slots % 8)[:, None, None] * 16 + d % 16
    return [(flat[at + 8 * head * i].double() - 128) * scales[base // 4 + i].double() for i in (0, 1)]


def _exact_blocks(cache, key, value, slots, head):
    """The blocks that get tokens, block by block and head by head as the definition
    says: {block: [keys, values]}, each [kv_heads, block, D]."""
    block = cache.shape[2] * 8
    order = np.argsort(slots.cpu().numpy() // block, kind="stable")
    ids = slots.cpu().numpy()[order] // block
    cuts = np.flatnonzero(np.diff(ids, prepend=-1))
    ends = np.append(cuts[1:], len(ids))
    every = torch.arange(block, device=cache.device)
    done = {}
    for c0, c1 in zip(cuts, ends):
        who = torch.from_numpy(order[c0:c1]).to(cache.device)
        b, off = int(ids[c0]), slots[who] % block
        held = _exact_read(cache, b * block + every, head)
        base = cache[b, :, 0].contiguous().view(torch.float32)[:, :2].double()
        out = []
        for i, x in enumerate((key, value)):
            x, y = x[who].double(), held[i].transpose(0, 1).clone()
            s = (x.abs().amax((0, 2)) / 127).float().double()
            if not bool((off == 0).any()):
                grown = s > base[:, i]
                s = torch.maximum(s, base[:, i])
                redone = torch.round(y / s.clamp(min=1e-300)[:, None, None]).clamp(-127, 127) * s[:, None, None]
                y = torch.where(grown[:, None, None], redone, y)
            t = s.clamp(min=1e-300)[:, None]
            y[:, off] = (torch.round(x / t).clamp(-127, 127) * s[:, None]).transpose(0, 1)
            out.append(y)
        done[b] = out
    return done


def _exact_evict(s):
    """Sequence by sequence: tables, weights, lengths and the ids that leave."""
    block, n_out = s["block"], []
    tables, weights = s["tables"].cpu().numpy().copy(), s["weights"].cpu().numpy().astype(np.float64)
    lens = s["lens"].cpu().numpy().astype(np.int64)
    ids = []
    for r, length in enumerate(lens):
        n = -(-int(length) // block)
        out = max(0, n - s["budget"])
        n_out.append(out)
        may = range(s["first"], n - s["last"])
        leave = sorted(sorted(may, key=lambda b: (weights[r, b], b))[:out])
        stay = np.setdiff1d(np.arange(n), leave)
        ids += [int(tables[r, b]) for b in leave]
        tables[r, :n] = tables[r, list(stay) + leave]
        weights[r, :n] = np.append(weights[r, stay], np.zeros(out))
    return tables, weights, lens - np.array(n_out) * block, np.array(n_out) * block, ids


def exact(case, seed):
    kind = case["kind"]
    s = prepare(case, seed)
    if kind == "rope":
        at = s["positions"] if s["shift"] is None else s["positions"] + s["shift"]
        return {n: torch.cat([_exact_rope(x, s[n + "_weight"], s["cos_sin"], p, case["interleaved"], s["eps"])
                              for x, p in zip(s[n].split(4096), at.split(4096))]) for n in ("query", "key")}
    if kind == "evict":
        weights = torch.from_numpy(_exact_evict(s)[1]).cuda()
        return {"tables": None, "weights": weights, "lens": None, "gone": None, "ring": None, "ring_state": None}
    head, block = case["head"], case["block"]
    if kind in ("write", "gather"):
        k, v = (torch.cat(x) for x in zip(*(_exact_read(s["cache"], p, head) for p in s["back"].split(8192))))
        if kind == "write":
            if len(s["slots"]) // block + case["requests"] > 8000:
                return None
            where = {}
            for i, slot in enumerate(s["back"].tolist()):
                where.setdefault(slot // block, []).append((i, slot % block))
            for b, kv in _exact_blocks(s["cache"], s["key"], s["value"], s["slots"], head).items():
                i, off = (torch.tensor(x, device="cuda") for x in zip(*where[b]))
                k[i], v[i] = kv[0][:, off].transpose(0, 1), kv[1][:, off].transpose(0, 1)
        return {"key": k, "value": v}
    group = case["heads"] // case["kv_heads"]
    weights = kind == "step" or case["weights"]
    done = {}
    if kind == "decode":
        tables, lens, query = s["tables"].cpu().numpy(), s["lens"].tolist(), s["query"].double()
        old = s["weights"].double() if weights else None
    else:
        tables, old, lens, gone, ids = _exact_evict(s)
        ring, (front, count) = s["ring"].cpu().numpy(), s["ring_state"].tolist()
        free = [int(ring[(front + i) % len(ring)]) for i in range(count)] + ids
        at = torch.from_numpy(lens + s["gone"].cpu().numpy() + gone).cuda()
        for r, n in enumerate(lens):
            if n % block == 0:
                tables[r, n // block] = free.pop(0)
        slots = torch.tensor([int(tables[r, n // block]) * block + n % block for r, n in enumerate(lens)],
                             device="cuda")
        raw = [_exact_rope(s["raw_" + x], s[x + "_weight"], s["cos_sin"], at, False, s["eps"])
               for x in ("query", "key")]
        dtype = TYPES[case["dtype"]]
        query = raw[0].to(dtype).double()
        done = _exact_blocks(s["cache"], raw[1].to(dtype), s["value"], slots, head)
        old, lens = torch.from_numpy(old).cuda(), [int(n) + 1 for n in lens]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    total = torch.zeros(tables.shape, dtype=torch.float64, device="cuda")
    tables = torch.from_numpy(np.ascontiguousarray(tables)).long().cuda()
    for r, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(n, device="cuda")
        k, v = _exact_read(s["cache"], tables[r][pos // block] * block + pos % block, head)
        last = int(tables[r, (n - 1) // block])
        if last in done:
            m = (n - 1) // block * block
            k[m:], v[m:] = (x[:, :n - m].transpose(0, 1) for x in done[last])
        w = torch.einsum("hgd,nhd->hgn", query[r].unflatten(0, (-1, group)), k) * float(s["scale"])
        w = torch.softmax(w, dim=-1)
        out[r] = torch.einsum("hgn,nhd->hgd", w, v).flatten(0, 1)
        if weights:
            w = torch.nn.functional.pad(w.sum((0, 1)), (0, -n % block)).view(-1, block).sum(-1)
            total[r, :len(w)] = DECAY * old[r, :len(w)] + w
    if kind == "decode":
        return {"out": out, "weights": total} if weights else {"out": out}
    return {"tables": None, "lens": None, "ring_state": None, "gone": None, "query": raw[0], "out": out,
            "weights": total}
