"""Cross attention and the operators of a block pool on the device: what is measured, on which cases, and their
plain forms.

An encoder-decoder model's decoder attends to its encoder's states at every layer and step, and is mostly decoded by
beam search: which beam goes on from which is known on the device only.  The states stand in the same kind of paged
cache as the decoder's own keys, and the pool's block tables, lengths and reference counts stand on the device.

  cross    every new token of a request attends to all of the request's stored keys (another length, no causal mask)
  fork     rows of the block tables become (prefixes of) other rows: whole blocks are shared, a shared partial last
           block gets a copy of its own; rows without a parent are freed.  With the K/V copies of every layer.
  grow     rows get room for new tokens, from the lowest free blocks on, and the tokens get their slots
  compact  live blocks move to the pool's lowest ids, and the tables follow.  With the K/V moves of every layer.
  copy     whole blocks copied in the caches of every layer
"""
import math
import random

import numpy as np
import torch

own = False  # True: the framework's operators; False: their plain forms

BS = 16                      # tokens per block
CROSS_WORKSPACE = 48 << 20   # what a serving program keeps for its cross attention calls


# ---------------------------------------------------------------- cases
def listed():
    gqa = {"heads": 32, "kv_heads": 8, "dim": 128}
    mha = {"heads": 32, "kv_heads": 32, "dim": 128}
    tiny = {"heads": 4, "kv_heads": 4, "dim": 64}
    return [
        # two short requests, one new token each: latency
        {"name": "cross_2_tiny", "op": "cross", "tokens": 1, "reqs": 2, "lo": 40, "hi": 300, "chunks": "", "lens": 1,
         **tiny},
        # a decoding batch, one token of each request, long documents
        {"name": "cross_48_gqa", "op": "cross", "tokens": 1, "reqs": 48, "lo": 256, "hi": 8192, "chunks": "",
         "lens": 2, **gqa},
        # beam search: four hypotheses of each of 64 requests share its encoder's states
        {"name": "cross_64_beams", "op": "cross", "tokens": 4, "reqs": 64, "lo": 512, "hi": 4096, "chunks": "",
         "lens": 3, **mha},
        # decoder prompts of odd sizes over documents of odd sizes, one of them empty
        {"name": "cross_prompts", "op": "cross", "tokens": 0, "reqs": 0, "lo": 0, "hi": 0,
         "chunks": "1999@9001,1203@2500,515@777,5@0", "lens": 4, **gqa},
        # one request of four beams in a small model
        {"name": "fork_4_tiny", "op": "fork", "groups": 1, "beams": 4, "prompt": 37, "hi": 30, "rollback": 0,
         "done": 0, "layers": 2, "pool": 48, "lens": 5, **tiny},
        # 32 requests of four beams, long prompts shared, every layer's K/V
        {"name": "fork_128_beams", "op": "fork", "groups": 32, "beams": 4, "prompt": 1000, "hi": 700, "rollback": 0,
         "done": 9, "layers": 32, "pool": 6000, "lens": 6, **gqa},
        # drafts verified: 48 requests are given room for up to 8 tokens more
        {"name": "grow_48", "op": "grow", "rows": 48, "lo": 256, "hi": 8192, "new": 8, "pool": 14000, "lens": 7, **gqa},
        # prompts of up to 2000 tokens admitted into a pool that is half full
        {"name": "grow_512", "op": "grow", "rows": 512, "lo": 0, "hi": 900, "new": 2000, "pool": 100000, "lens": 8,
         **gqa},
        # a small model's pool
        {"name": "compact_8_tiny", "op": "compact", "rows": 8, "lo": 16, "hi": 400, "pool": 333, "fill": 0.6,
         "layers": 2, "lens": 9, **tiny},
        # a serving pool of 28,610 blocks (60 GB over 32 layers) after many requests came and went, two layers' worth
        {"name": "compact_256_gqa", "op": "compact", "rows": 256, "lo": 256, "hi": 2500, "pool": 28610, "fill": 0.9,
         "layers": 2, "lens": 10, **gqa},
        # the blocks that a scheduling step copies on write, every layer of an 8-bit cache
        {"name": "copy_24_fp8", "op": "copy", "pairs": 24, "pool": 300, "layers": 32, "bits": 8, "lens": 11, **gqa},
        # 1024 blocks (16,384 tokens) of every layer
        {"name": "copy_1024_gqa", "op": "copy", "pairs": 1024, "pool": 2100, "layers": 32, "bits": 16, "lens": 12, **gqa},
    ]


SHAPES = [(32, 8, 128), (32, 32, 128), (32, 1, 128), (32, 2, 128), (16, 8, 128), (64, 8, 128), (12, 12, 128),
          (24, 6, 128), (4, 4, 64), (8, 4, 64), (32, 8, 64), (40, 5, 64)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hk, a = rng.choice(SHAPES)
    c = {"heads": hq, "kv_heads": hk, "dim": a}
    op = rng.choice(["cross", "cross", "cross", "fork", "grow", "compact", "copy"])
    lens = rng.randrange(1 << 20)
    block = hk * BS * a * 4                                             # K and V bytes of one layer's block, bf16
    if op == "cross":
        t = rng.choice([0, 1, 1, 1, rng.randint(2, 9)])
        reqs = hi = 0
        chunks = ""
        if t:
            reqs = _log(rng, 1, 200)
            hi = _log(rng, 20, int(min(16384, 3e5 * 8 / (reqs * max(hk, hq * t / 8)))) + 20)
        if not t or rng.random() < 0.2:
            parts = []
            for i in range(rng.choice([1, 1, 2, 3])):
                keys = [_log(rng, 1, 8000), _log(rng, 1, 8000), 0 if i else 4000]
                parts.append("%d@%d" % (_log(rng, 1, 1500), rng.choice(keys)))
            chunks = ",".join(parts)
        return {"op": op, "tokens": t, "reqs": reqs, "lo": rng.choice([0, hi // 3]), "hi": hi, "chunks": chunks,
                "lens": lens, **c}
    if op == "fork":
        groups, beams = _log(rng, 1, 64), rng.randint(1, 8)
        prompt, hi = _log(rng, 1, 2000), _log(rng, 1, 600)
        need = groups * (prompt // BS + 1 + beams * (hi // BS + 4)) + 2
        return {"op": op, "groups": groups, "beams": beams, "prompt": prompt, "hi": hi, "rollback": rng.choice([0, 0, 5]),
                "done": rng.choice([0, 3, 7]), "layers": max(1, min(32, int(1e10 / (need * block)))), "pool": need + 7,
                "lens": lens, **c}
    if op == "grow":
        rows = _log(rng, 1, 512)
        hi, new = _log(rng, 1, 4000), _log(rng, 1, 2000)
        return {"op": op, "rows": rows, "lo": 0, "hi": hi, "new": new, "lens": lens,
                "pool": int(rows * (hi + new + 40) / BS * rng.choice([1.0, 1.5])) + 3, **c}
    if op == "compact":
        rows, hi = _log(rng, 1, 256), _log(rng, 16, 2500)
        fill = rng.choice([0.3, 0.6, 0.9])
        pool = int(rows * (hi / BS + 2) / fill) + 3
        return {"op": op, "rows": rows, "lo": 0, "hi": hi, "pool": pool, "fill": fill, "lens": lens,
                "layers": max(1, min(32, int(3e9 / (pool * block)))), **c}
    layers = rng.choice([1, 7, 32])
    bits = rng.choice([8, 16])
    pairs = _log(rng, 1, max(1, min(1024, int(4e9 * 16 / bits / (2 * layers * block)))))
    return {"op": op, "pairs": pairs, "pool": 2 * pairs + 9, "layers": layers, "bits": bits, "lens": lens, **c}


def _blocks(n):
    return -(-n // BS)


def _cross_lengths(case):
    """(new tokens, stored keys) of every request: the short ones first, then the prompts."""
    r = random.Random(case["lens"])
    reqs = [(case["tokens"], r.randint(case["lo"], case["hi"])) for _ in range(case["reqs"])]
    for part in filter(None, case["chunks"].split(",")):
        q, n = part.split("@")
        reqs.append((int(q), int(n)))
    return reqs


def _fork_plan(case):
    """Lengths, parents and kept lengths (-1: all) of every row."""
    r = np.random.RandomState(case["lens"])
    g, b = case["groups"], case["beams"]
    lens = np.repeat(case["prompt"] + r.randint(0, case["hi"] + 1, g), b)
    # beams go on from a few of their group: the better ones more often
    parents = (np.arange(g)[:, None] * b + np.minimum(r.geometric(0.45, (g, b)) - 1, b - 1)).reshape(-1)
    if case["done"]:
        parents.reshape(g, b)[case["done"] - 1::case["done"]] = -1       # these requests have ended
    keep = lens - r.randint(0, case["rollback"] + 1, g * b) if case["rollback"] else np.full(g * b, -1)
    return lens, parents, np.maximum(keep, -1)


def _grow_plan(case):
    r = np.random.RandomState(case["lens"])
    lens = r.randint(case["lo"], case["hi"] + 1, case["rows"])
    return lens, r.randint(0, case["new"] + 1, case["rows"])


def _compact_lens(case):
    """Row lengths that fill the pool as far as the case says, at most."""
    r = np.random.RandomState(case["lens"])
    lens = r.randint(case["lo"], case["hi"] + 1, case["rows"])
    return np.where(np.cumsum(_blocks(lens)) <= case["fill"] * case["pool"], lens, 0)


# ---------------------------------------------------------------- inputs
def _rows(gen, shape, channel, token_spread):
    """bf16 rows [..., heads, dim]: normal values, a spread of the channels'
    sizes with a few large ones (as keys have), tokens of different size."""
    y = torch.randn(shape, device="cuda", generator=gen)
    t = torch.randn((*shape[:-2], 1, 1), device="cuda", generator=gen)
    return (y * channel * torch.exp(token_spread * t)).to(torch.bfloat16)


def _bits(gen, shape, dtype):
    """A cache of `shape`: random values."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=dtype, device="cuda")
    for lo in range(0, n, 1 << 28):
        m = min(1 << 28, n - lo)
        if dtype == torch.uint8:
            out[lo:lo + m] = torch.randint(100, 140, (m,), device="cuda", generator=gen, dtype=torch.uint8)
        else:
            out[lo:lo + m] = torch.randn(m, device="cuda", generator=gen, dtype=torch.bfloat16).to(dtype)
    return out.view(shape)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _caches(case, gen):
    """K and V of every layer [layers, blocks, Hkv, 16, A], in 8 bits with their rows' exponents."""
    shape = (case["layers"], case["pool"], case["kv_heads"], BS, case["dim"])
    if case.get("bits") == 8:
        return [_bits(gen, shape, torch.float8_e4m3fn), _bits(gen, shape, torch.float8_e4m3fn),
                _bits(gen, shape[:-1], torch.uint8), _bits(gen, shape[:-1], torch.uint8)]
    return [_bits(gen, shape, torch.bfloat16), _bits(gen, shape, torch.bfloat16)]


def _fill_tables(lens, ids, width):
    """Block tables of rows that share nothing; ids in order of use."""
    tables = np.full((len(lens), width), -1, np.int32)
    at = 0
    for r, n in enumerate(_blocks(lens)):
        tables[r, :n] = ids[at:at + n]
        at += n
    return tables


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.RandomState(seed % (1 << 31))
    op = case["op"]
    s = {"op": op}
    if op == "cross":
        hq, hk, a = case["heads"], case["kv_heads"], case["dim"]
        reqs = _cross_lengths(case)
        q_lens, kv = np.array([q for q, _ in reqs]), np.array([n for _, n in reqs])
        nb = int(_blocks(kv).sum()) + int(_blocks(kv).sum()) // 8 + 2
        tables = _fill_tables(kv, host.permutation(nb), max(1, int(_blocks(kv).max())))
        cu = np.concatenate([[0], np.cumsum(q_lens)])
        channel = torch.exp(0.4 * torch.randn(hk, 1, a, device="cuda", generator=gen))
        channel[:, :, 3] *= 5
        s["q"] = _rows(gen, (int(cu[-1]), hq, a), 1.0, 0.2)
        for name, ch in (("k", channel), ("v", 1.0)):
            s[name] = torch.empty(nb, hk, BS, a, dtype=torch.bfloat16, device="cuda")
            step = max(1, (1 << 26) // (hk * BS * a))
            for lo in range(0, nb, step):
                s[name][lo:lo + step] = _rows(gen, (min(step, nb - lo), hk, BS, a), ch, 0.1)
        s["out"] = torch.empty_like(s["q"])
        s["cu"], s["kv_lens"], s["tables"] = _ints(cu), _ints(kv), _ints(tables)
        s["scale"] = 1.0 / math.sqrt(a)
        s["max_q"], s["max_kv"] = int(q_lens.max()), max(1, int(kv.max()))
        s["short"], s["tokens"] = case["reqs"], case["tokens"]          # requests with few tokens come first
        s["short_kv"] = max(1, int(kv[:case["reqs"]].max())) if case["reqs"] else 0
        s["workspace"] = torch.empty(CROSS_WORKSPACE, dtype=torch.uint8, device="cuda")
        return s
    pool = case["pool"]
    ids = host.permutation(pool)
    if op == "copy":
        s["caches"] = _caches(case, gen)
        s["pairs"] = _ints(ids[:2 * case["pairs"]].reshape(-1, 2))
        return s
    if op == "fork":
        lens, parents, keep = _fork_plan(case)
        b, shared = case["beams"], case["prompt"] // BS
        own_blocks = _blocks(lens) - shared
        width = int(_blocks(lens).max()) + 1
        tables = np.full((len(lens), width), -1, np.int32)
        at = 0
        for r in range(len(lens)):
            if r % b == 0:
                first = ids[at:at + shared]
                at += shared
            tables[r, :shared] = first
            tables[r, shared:shared + own_blocks[r]] = ids[at:at + own_blocks[r]]
            at += own_blocks[r]
        s["parents"], s["keep"] = _ints(parents), _ints(keep)
        s["pairs"] = _ints(np.zeros((len(lens), 2)))
    elif op == "grow":
        lens, new = _grow_plan(case)
        tables = _fill_tables(lens, ids, int(_blocks(lens + new).max()) + 1)
        s["cu"] = _ints(np.concatenate([[0], np.cumsum(new)]))
        s["ctx"] = _ints(np.zeros(len(lens)))
        s["slots"] = torch.zeros(int(new.sum()), dtype=torch.int64, device="cuda")
    else:
        lens = _compact_lens(case)
        tables = _fill_tables(lens, ids, int(_blocks(lens).max()) + 1)
        for r in range(4, len(lens), 5):                                # some share a prefix with the row before
            n = int(min(lens[r], lens[r - 1]) // BS)
            tables[r, :n] = tables[r - 1, :n]
        s["block_map"] = _ints(np.zeros(pool))
        s["pairs"] = _ints(np.zeros((pool // 2 + 1, 2)))
        s["counts"] = _ints(np.zeros(2))
    refs = np.bincount(tables[tables >= 0], minlength=pool)
    # one buffer: tables, lengths and reference counts, and what they were at first
    s["first"] = _ints(np.concatenate([tables.reshape(-1), lens, refs]))
    s["pool"] = s["first"].clone()
    n, w = tables.shape
    s["tables"] = s["pool"][:n * w].view(n, w)
    s["lens"], s["refs"] = s["pool"][n * w:n * w + n], s["pool"][n * w + n:]
    s["workspace"] = torch.empty(n * w * 4 + pool * 12 + (1 << 20), dtype=torch.uint8, device="cuda")
    if op != "grow":
        s["caches"] = _caches(case, gen)
    return s


# ---------------------------------------------------------------- plain forms
def _attend(s, first, count, max_q, max_kv):
    """Requests first .. first + count - 1 as one padded batch: fp32 outputs of
    their tokens, [count, max_q, Hq, A]; a request without keys gives zeros."""
    hq, a = s["q"].shape[1:]
    hk = s["k"].shape[1]
    cu, kv = s["cu"][first:first + count + 1].long(), s["kv_lens"][first:first + count].long()
    blocks = s["tables"][first:first + count, :_blocks(max_kv)].long().clamp(min=0)
    seen = torch.arange(blocks.shape[1] * BS, device="cuda") < kv[:, None]
    k = s["k"][blocks].float().transpose(1, 2).reshape(count, hk, -1, a)          # [R, Hkv, keys, A]
    v = s["v"][blocks].float().transpose(1, 2).reshape(count, hk, -1, a)
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    tokens = (cu[:-1, None] + torch.arange(max_q, device="cuda")).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[tokens]                                                     # [R, m, Hq, A]
    q = q.view(count, max_q, hk, hq // hk, a).permute(0, 2, 3, 1, 4).reshape(count, hk, -1, a)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]                            # [R, Hkv, G * m, keys]
    x = x.masked_fill(~seen[:, None, None, :], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    o = torch.where((kv > 0)[:, None, None, None], o, 0.0)
    return o.view(count, hk, hq // hk, max_q, a).permute(0, 3, 1, 2, 4).reshape(count, max_q, hq, a)


def _cross(s):
    d, n = s["short"], s["kv_lens"].shape[0]
    out = torch.empty_like(s["q"])
    if d:
        out[:d * s["tokens"]] = _attend(s, 0, d, s["tokens"], s["short_kv"]).flatten(0, 1).to(out.dtype)
    if n > d:
        o = _attend(s, d, n - d, s["max_q"], s["max_kv"])
        cu = s["cu"][d:].long()
        t = torch.arange(d * s["tokens"], out.shape[0], device="cuda")
        r = torch.searchsorted(cu, t, right=True) - 1
        out[d * s["tokens"]:] = o[r, t - cu[r]].to(out.dtype)
    return out


def _count(ids, mask, pool):
    """How often each block stands among the masked entries."""
    at = torch.where(mask & (ids >= 0), ids.long(), pool).reshape(-1)
    return torch.zeros(pool + 1, dtype=torch.int64, device="cuda").index_add_(0, at, torch.ones_like(at))[:pool]


def _free_blocks(refs):
    """Block ids, the free ones first, from the lowest on, and their number."""
    return torch.argsort(refs > 0, stable=True), (refs == 0).sum()


def _fork(s):
    tables, lens, refs = s["tables"], s["lens"], s["refs"]
    n, width = tables.shape
    pool = refs.shape[0]
    col, row = torch.arange(width, device="cuda"), torch.arange(n, device="cuda")
    parents = s["parents"].long()
    old, was = tables.clone(), lens.long()
    have = torch.where(parents >= 0, was[parents.clamp(min=0)], 0)
    keep = torch.where(s["keep"] < 0, have, torch.minimum(s["keep"].long(), have))
    before, after = col < -(-was // BS)[:, None], col < -(-keep // BS)[:, None]
    new = torch.where(after, old[parents.clamp(min=0)], torch.where(before, -1, old))
    count = refs.long() + _count(new, after, pool) - _count(old, before, pool)
    # a partial last block stays with its lowest row if nothing else holds it
    last = (-(-keep // BS) - 1).clamp(min=0)
    block = new[row, last].long()
    part = (keep % BS != 0) & (block >= 0)
    at = torch.where(part, block, pool)
    holders = torch.zeros(pool + 1, dtype=torch.int64, device="cuda").index_add_(0, at, torch.ones_like(at))
    lowest = torch.full((pool + 1,), n, device="cuda").scatter_reduce_(0, at, row, "amin")
    need = part & ~((count[block.clamp(min=0)] == holders[at]) & (lowest[at] == row))
    ids, free = _free_blocks(count)
    rank = need.long().cumsum(0) - 1
    got = need & (rank < free)
    fresh = ids[rank.clamp(min=0, max=pool - 1)]
    keep = torch.where(need & ~got, keep // BS * BS, keep)
    new[row, last] = torch.where(need, torch.where(got, fresh, -1), new[row, last].long()).to(new.dtype)
    ends = torch.zeros(pool + 1, dtype=torch.int64, device="cuda")
    ends.index_add_(0, torch.where(need, block, pool), -torch.ones_like(row))
    ends.index_add_(0, torch.where(got, fresh, pool), torch.ones_like(row))
    tables.copy_(new)
    lens.copy_(keep)
    refs.copy_(count + ends[:pool])
    s["pairs"].copy_(torch.where(got[:, None], torch.stack([block, fresh], 1), -1))


def _grow(s):
    tables, lens, refs = s["tables"], s["lens"], s["refs"]
    n, width = tables.shape
    pool = refs.shape[0]
    cu, was = s["cu"].long(), lens.long()
    now = was + cu[1:] - cu[:-1]
    had, have = -(-was // BS), -(-now // BS)
    need = have - had
    ids, free = _free_blocks(refs)
    end = need.cumsum(0)
    ok = (need == 0) | (end <= free)
    col = torch.arange(width, device="cuda")
    new = (col >= had[:, None]) & (col < have[:, None]) & ok[:, None]
    rank = (end - need - had)[:, None] + col
    tables.copy_(torch.where(new, ids[rank.clamp(min=0, max=pool - 1)], tables.long()))
    refs.add_(_count(tables, new, pool).to(refs.dtype))
    s["ctx"].copy_(was)
    lens.copy_(torch.where(ok, now, was))
    t = torch.arange(s["slots"].shape[0], device="cuda")
    r = torch.searchsorted(cu, t, right=True) - 1
    pos = was[r] + t - cu[r]
    slot = tables[r, (pos // BS).clamp(max=width - 1)].long() * BS + pos % BS
    s["slots"].copy_(torch.where(ok[r], slot, -1))


def _compact(s):
    tables, lens, refs = s["tables"], s["lens"], s["refs"]
    pool, most = refs.shape[0], s["pairs"].shape[0]
    ids = torch.arange(pool, device="cuda")
    live = refs > 0
    n_live = live.sum()
    hole, moves = ~live & (ids < n_live), live & (ids >= n_live)
    rank = moves.long().cumsum(0) - 1
    to = torch.argsort(~hole, stable=True)[rank.clamp(min=0)]
    block_map = torch.where(moves, to, torch.where(live, ids, -1))
    pairs = torch.full((most + 1, 2), -1, dtype=torch.int64, device="cuda")
    pairs[torch.where(moves, rank, most)] = torch.stack([ids, to], 1)
    after = torch.zeros(pool + 1, dtype=torch.int64, device="cuda")
    after[torch.where(live, block_map, pool)] = refs.long()
    held = (torch.arange(tables.shape[1], device="cuda") < -(-lens.long() // BS)[:, None]) & (tables >= 0)
    tables.copy_(torch.where(held, block_map[tables.long().clamp(min=0)], tables.long()))
    refs.copy_(after[:pool])
    s["block_map"].copy_(block_map)
    s["pairs"].copy_(pairs[:most])
    s["counts"].copy_(torch.stack([n_live, moves.sum()]))


def _copy(s):
    kept = s["pairs"][s["pairs"][:, 0] >= 0].long()
    src, dst = kept[:, 0], kept[:, 1]
    s["caches"][0].view(torch.uint8)[:, dst] = s["caches"][0].view(torch.uint8)[:, src]
    s["caches"][1].view(torch.uint8)[:, dst] = s["caches"][1].view(torch.uint8)[:, src]
    if len(s["caches"]) == 4:
        s["caches"][2][:, dst] = s["caches"][2][:, src]
        s["caches"][3][:, dst] = s["caches"][3][:, src]


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if op in ("grow", "compact"):
        s["pool"].copy_(s["first"])                                     # the pool as it was before the step
    if own:
        import paged_kv_cache_cb_gb300 as cb
        if op == "cross":
            cb.cb_paged_cross_attention(s["q"], s["cu"], s["kv_lens"], s["tables"], s["k"], s["v"], s["out"],
                                        s["scale"], s["workspace"], s["max_q"], s["max_kv"])
            return {"out": s["out"]}
        if op == "fork":
            cb.cb_fork_blocks(s["parents"], s["keep"], s["tables"], s["lens"], s["refs"], s["pairs"], s["workspace"])
        elif op == "grow":
            cb.cb_grow_blocks(s["cu"], s["tables"], s["lens"], s["refs"], s["ctx"], s["slots"], s["workspace"])
        elif op == "compact":
            cb.cb_compact_blocks(s["tables"], s["lens"], s["refs"], s["block_map"], s["pairs"], s["counts"],
                                 s["workspace"])
        if op != "grow":
            cb.cb_copy_blocks_layers(s["pairs"], s["caches"])
    else:
        if op == "cross":
            return {"out": _cross(s)}
        if op == "fork":
            _fork(s)
        elif op == "grow":
            _grow(s)
        elif op == "compact":
            _compact(s)
        if op != "grow":
            _copy(s)
    if op == "copy":
        return {"caches": s["caches"]}
    res = {"tables": s["tables"], "lens": s["lens"], "refs": s["refs"]}
    if op == "fork":
        return {"pairs": s["pairs"], "caches": s["caches"], **res}
    if op == "grow":
        return {"ctx": s["ctx"], "slots": s["slots"], **res}
    return {"block_map": s["block_map"], "pairs": s["pairs"], "counts": s["counts"], "caches": s["caches"], **res}


def work(case):
    hq, hk, a = case["heads"], case["kv_heads"], case["dim"]
    op = case["op"]
    if op == "cross":
        reqs = _cross_lengths(case)
        tokens, keys = sum(q for q, _ in reqs), sum(n for q, n in reqs if q)
        return {"bytes": keys * hk * a * 4 + tokens * hq * a * 4, "flops": 4 * a * hq * sum(q * n for q, n in reqs)}
    if op == "copy":
        row = 2 * a if case["bits"] == 16 else a + 1
        return {"bytes": case["pairs"] * (8 + case["layers"] * 2 * 2 * hk * BS * row), "flops": 0}
    block = case["layers"] * 2 * hk * BS * 2 * a if op != "grow" else 0     # K and V of a block in every layer
    if op == "grow":
        lens, new = _grow_plan(case)
        need = int((_blocks(lens + new) - _blocks(lens)).sum())
        # lengths and offsets, the free blocks' counts read and written, tables and slots written
        return {"bytes": 16 * len(lens) + 12 * need + 8 * int(new.sum()), "flops": 0}
    if op == "fork":
        lens, parents, keep = _fork_plan(case)
        have = np.where(parents >= 0, lens[parents], 0)
        keep = np.where(keep < 0, have, np.minimum(keep, have))
        moved = parents != np.arange(len(lens))
        # changed rows' entries: the parent's read, the row's own read and written, both blocks' counts read and written
        ints = int((3 * _blocks(np.maximum(keep, lens)) + 4 * _blocks(keep))[moved].sum()) + 8 * len(lens)
        kept = len(set(parents[(parents >= 0) & (keep % BS != 0)]))
        copies = int(((parents >= 0) & (keep % BS != 0)).sum()) - kept
        return {"bytes": 4 * ints + copies * block * 2, "flops": 0}
    lens = _compact_lens(case)
    n = _blocks(lens)
    live = int(n.sum())
    for r in range(4, len(lens), 5):
        live -= int(min(lens[r], lens[r - 1]) // BS)
    moves = live * (case["pool"] - live) / case["pool"]                     # blocks above the line, at random places
    return {"bytes": 4 * (3 * case["pool"] + 2 * int(n.sum())) + moves * (8 + block * 2), "flops": 0}


# ---------------------------------------------------------------- the same in 64 bits
def exact(case, seed):
    if case["op"] != "cross" or work(case)["flops"] > 1.2e13:
        return None                                                     # the others move what they are given
    s = prepare(case, seed)
    hq, hk, a = case["heads"], case["kv_heads"], case["dim"]
    g, out, t = hq // hk, torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for r, (q, n) in enumerate(_cross_lengths(case)):
        if q and n:
            blk = s["tables"][r, :_blocks(n)].long()
            for h in range(hk):
                k, v = (s[name][blk, h].reshape(-1, a)[:n].double() for name in ("k", "v"))
                x = torch.einsum("qgd,nd->gqn", s["q"][t:t + q, h * g:(h + 1) * g].double(), k) / math.sqrt(a)
                out[t:t + q, h * g:(h + 1) * g] = torch.einsum("gqn,nd->qgd", torch.softmax(x, -1), v)
        t += q
    return {"out": out}
