"""Operators of the 8-bit KV cache: what is measured, on which cases, and their plain forms.

The cache holds K and V as e4m3 values with one power-of-two exponent per row
(token, KV head): a row x is stored as round_e4m3(x * 2^-e) and the byte e + 127,
e being the least integer >= -126 with max|x| <= 448 * 2^e.  A row that holds a
NaN or an infinity is stored as zeros with the byte 255 and stands for NaNs.

  append   new K/V rows quantised and written to their slots
  gather   stored rows read back as bf16
  decode   one new token per request attends over its stored keys
  chunk    several new tokens per request attend to the stored keys and,
           causally, to each other
  step     append, then attention of a ragged batch of both kinds (one call)
"""
import math
import random

import numpy as np
import torch

own = False  # True: the framework's operators; False: their plain forms

BS = 16                      # tokens per block
WORKSPACE = 128 << 20        # what a serving program keeps for its attention calls


# ---------------------------------------------------------------- cases
def listed():
    gqa = {"heads": 32, "kv_heads": 8, "dim": 128}
    mha = {"heads": 32, "kv_heads": 32, "dim": 128}
    mqa = {"heads": 32, "kv_heads": 1, "dim": 128}
    tiny = {"heads": 4, "kv_heads": 4, "dim": 64}
    return [
        # the append of a step of 48 decoding requests: latency
        {"name": "append_48_gqa", "op": "append", "tokens": 48, "skip": 0, **gqa},
        # a padded batch of an odd number of tokens: some have no slot
        {"name": "append_1073_mha", "op": "append", "tokens": 1073, "skip": 7, **mha},
        # a whole padded prefill of 8 prompts of 8192 tokens
        {"name": "append_65536_gqa", "op": "append", "tokens": 65536, "skip": 0, **gqa},
        # one short request's rows read back (moved to another cache)
        {"name": "gather_333_tiny", "op": "gather", "tokens": 333, "skip": 5, **tiny},
        # a long prompt's rows read back
        {"name": "gather_32768_gqa", "op": "gather", "tokens": 32768, "skip": 0, **gqa},
        # the tail of a serving trace: two requests still decoding
        {"name": "decode_2_gqa", "op": "decode", "decodes": 2, "lo": 4800, "hi": 5000, "lens": 1, "window": 0, **gqa},
        # the decodes of the mixed serving step
        {"name": "decode_48_gqa", "op": "decode", "decodes": 48, "lo": 256, "hi": 8192, "lens": 2, "window": 0, **gqa},
        # a layer without grouped heads
        {"name": "decode_64_mha", "op": "decode", "decodes": 64, "lo": 512, "hi": 4096, "lens": 3, "window": 0, **mha},
        # many long requests on a single KV head
        {"name": "decode_256_mqa", "op": "decode", "decodes": 256, "lo": 1024, "hi": 16384, "lens": 4, "window": 0,
         **mqa},
        # two prompts' chunks of odd sizes after stored prefixes, under a rolling window
        {"name": "chunk_2_window", "op": "chunk", "chunks": "301@2500,512@1024", "lens": 5, "window": 1000, **gqa},
        # a long prompt's chunk after 30,720 stored tokens
        {"name": "chunk_2048_long", "op": "chunk", "chunks": "2048@30720", "lens": 6, "window": 0, **gqa},
        # a serving step: 48 decodes and two prefill chunks, with the append
        {"name": "step_mixed", "op": "step", "decodes": 48, "lo": 256, "hi": 8192, "chunks": "512@1024,512@2048",
         "lens": 7, "window": 0, **gqa},
    ]


SHAPES = [(32, 8, 128), (32, 32, 128), (32, 1, 128), (32, 2, 128), (16, 8, 128), (64, 8, 128), (12, 12, 128),
          (24, 6, 128), (4, 4, 64), (8, 4, 64), (32, 8, 64), (40, 5, 64)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hk, a = rng.choice(SHAPES)
    c = {"heads": hq, "kv_heads": hk, "dim": a}
    op = rng.choice(["append", "gather", "decode", "decode", "chunk", "step"])
    if op in ("append", "gather"):
        return {"op": op, "tokens": _log(rng, 1, 65536 * 8 // max(8, hk)), "skip": rng.choice([0, 0, 3, 11]), **c}
    window = rng.choice([0, 0, 0, 16, _log(rng, 17, 4000)])
    lens = rng.randrange(1 << 20)
    n, hi, chunks = 0, 0, ""
    if op in ("decode", "step"):
        n = _log(rng, 1, 200)
        most = int(min(16384, 3e5 * 8 / (n * max(hk, hq / 8))))      # stored rows in all
        hi = _log(rng, min(40, most), most)
    if op in ("chunk", "step"):
        parts = []
        for _ in range(rng.choice([1, 1, 2, 3])):
            q = _log(rng, 2, 1500)
            parts.append("%d@%d" % (q, rng.choice([0, _log(rng, 1, 6000)])))
        chunks = ",".join(parts)
    return {"op": op, "decodes": n, "lo": rng.choice([0, hi // 3]), "hi": hi, "chunks": chunks, "lens": lens,
            "window": window, **c}


def _lengths(case):
    """(q_len, ctx) of every request: the decodes first, then the chunks."""
    r = random.Random(case["lens"])
    reqs = [(1, r.randint(case["lo"], case["hi"])) for _ in range(case.get("decodes", 0))]
    for part in filter(None, case.get("chunks", "").split(",")):
        q, ctx = part.split("@")
        reqs.append((int(q), int(ctx)))
    return reqs


# ---------------------------------------------------------------- inputs
def _rows(gen, n, heads, dim, channel, token_spread):
    """bf16 rows [n, heads, dim]: normal values, a spread of the channels'
    sizes with a few large ones (as keys have), tokens of different size."""
    x = torch.empty(n, heads, dim, device="cuda", dtype=torch.bfloat16)
    for lo in range(0, n, 65536):
        y = torch.randn(min(65536, n - lo), heads, dim, device="cuda", generator=gen)
        t = torch.randn(y.shape[0], 1, 1, device="cuda", generator=gen)
        x[lo:lo + 65536] = y * channel * torch.exp(token_spread * t)
    return x


def _channels(gen, heads, dim):
    c = torch.exp(0.4 * torch.randn(heads, dim, device="cuda", generator=gen))
    c[:, 3] *= 5
    c[:, dim // 2 + 5] *= 4
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.RandomState(seed % (1 << 31))
    hq, hk, a = case["heads"], case["kv_heads"], case["dim"]
    s = {"op": case["op"]}
    kch = _channels(gen, hk, a)
    if case["op"] in ("append", "gather"):
        n = case["tokens"]
        nb = -(-n // BS) + 2
        slots = host.permutation(nb * BS)[:n].astype(np.int64) if n < 4096 else np.concatenate(
            [b * BS + np.arange(BS) for b in host.permutation(nb)])[:n].astype(np.int64)
        if case["skip"]:
            slots[::case["skip"]] = -1
        s["slots"] = torch.from_numpy(slots).cuda()
    else:
        reqs = _lengths(case)
        blocks = [-(-(q + c) // BS) for q, c in reqs]
        nb = sum(blocks) + sum(blocks) // 8 + 2
        order = host.permutation(nb).astype(np.int32)
        tables = np.full((len(reqs), max(blocks)), -1, np.int32)
        at = 0
        for r, b in enumerate(blocks):
            tables[r, :b] = order[at:at + b]
            at += b
        q_lens = np.array([q for q, _ in reqs], np.int32)
        ctx = np.array([c for _, c in reqs], np.int32)
        cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        n = int(cu[-1])
        s["cu"], s["ctx"] = torch.from_numpy(cu).cuda(), torch.from_numpy(ctx).cuda()
        s["tables"] = torch.from_numpy(tables).cuda()
        s["q"] = _rows(gen, n, hq, a, 1.0, 0.2)
        s["scale"] = 1.0 / math.sqrt(a)
        s["window"] = case["window"]
        s["max_q"], s["max_kv"] = int(q_lens.max()), int((q_lens + ctx).max())
        s["decodes"] = int((q_lens == 1).sum())                    # the first requests of the batch
        s["max_decode_kv"] = int((ctx + 1)[q_lens == 1].max()) if s["decodes"] else 0
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        if case["op"] == "step":
            slots = np.concatenate([tables[r, (c + np.arange(q)) // BS].astype(np.int64) * BS + (c + np.arange(q)) % BS
                                    for r, (q, c) in enumerate(reqs)])
            s["slots"] = torch.from_numpy(slots).cuda()
    if case["op"] in ("append", "step"):
        s["k_new"], s["v_new"] = _rows(gen, n, hk, a, kch, 0.1), _rows(gen, n, hk, a, 1.0, 0.5)
    for name, channel, spread in (("k", kch, 0.1), ("v", 1.0, 0.5)):
        if case["op"] == "append":                                 # an empty cache
            s[name] = torch.zeros(nb, hk, BS, a, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            s[name + "_exps"] = torch.zeros(nb, hk, BS, dtype=torch.uint8, device="cuda")
            continue
        s[name] = torch.empty(nb, hk, BS, a, dtype=torch.float8_e4m3fn, device="cuda")
        s[name + "_exps"] = torch.empty(nb, hk, BS, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (hk * BS * a))
        for lo in range(0, nb, step):
            m = min(step, nb - lo)
            values, exps = _quantise(_rows(gen, m * BS, hk, a, channel, spread))
            s[name][lo:lo + m] = values.view(m, BS, hk, a).transpose(1, 2)
            s[name + "_exps"][lo:lo + m] = exps.view(m, BS, hk).transpose(1, 2)
    if case["op"] == "gather":
        s["k_out"] = torch.zeros(n, hk, a, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(n, hk, a, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _power(e):
    """2^e in fp32 for integers e in [-126, 127], from its bits (exact)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """bf16 rows [..., A] -> (e4m3 values, exponent bytes)."""
    f = x.float()
    largest = f.abs().amax(-1)
    part, power = torch.frexp(largest)                   # largest = part * 2^power, 1/2 <= part < 1; 448 = 7/8 * 2^9
    e = torch.where(part <= 0.875, power - 9, power - 8).clamp(min=-126)
    e = torch.where(largest > 0, e, -126)
    bad = ~torch.isfinite(f).all(-1)
    y = f * _power(-torch.where(bad, 0, e))[..., None]
    y = torch.where(bad[..., None], 0.0, y)
    return y.to(torch.float8_e4m3fn), torch.where(bad, 255, e + 127).to(torch.uint8)


def _values(rows, exps):
    """e4m3 rows and their exponent bytes -> fp32 values."""
    e = exps.to(torch.int32)
    f = torch.where(e == 255, float("nan"), _power((e - 127).clamp(min=-126)))
    return rows.float() * f[..., None]


def _write(cache, exps, slots, rows):
    values, e = _quantise(rows)
    kept = slots >= 0
    at = slots[kept]
    cache.view(torch.uint8)[at // BS, :, at % BS] = values.view(torch.uint8)[kept]
    exps[at // BS, :, at % BS] = e[kept]


def _read(cache, exps, slots, out):
    kept = slots >= 0
    at = slots[kept]
    rows = cache.view(torch.uint8)[at // BS, :, at % BS].view(torch.float8_e4m3fn)
    out[kept] = _values(rows, exps[at // BS, :, at % BS]).to(out.dtype)


def _attend(s, first, count, max_q, max_kv):
    """Requests first .. first + count - 1 as one padded batch: fp32 outputs of
    their tokens, [count, max_q, Hq, A]."""
    hq, a = s["q"].shape[1:]
    hk = s["k"].shape[1]
    cu, ctx = s["cu"][first:first + count + 1].long(), s["ctx"][first:first + count].long()
    blocks = s["tables"][first:first + count, :-(-max_kv // BS)].long().clamp(min=0)
    k = _values(s["k"].view(torch.uint8)[blocks].view(torch.float8_e4m3fn), s["k_exps"][blocks])
    v = _values(s["v"].view(torch.uint8)[blocks].view(torch.float8_e4m3fn), s["v_exps"][blocks])
    k = k.transpose(1, 2).reshape(count, hk, -1, a)                  # [R, Hkv, keys, A]
    v = v.transpose(1, 2).reshape(count, hk, -1, a)
    i = torch.arange(max_q, device="cuda")
    tokens = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[tokens]                                       # [R, m, Hq, A]
    q = q.view(count, max_q, hk, hq // hk, a).permute(0, 2, 3, 1, 4).reshape(count, hk, -1, a)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]              # [R, Hkv, G * m, keys]
    pos = (ctx[:, None] + i)[..., None]                              # [R, m, 1]
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key <= pos) & (key > pos - s["window"] if s["window"] else key >= 0)
    seen = seen[:, None, None].expand(count, 1, hq // hk, max_q, -1).reshape(count, 1, -1, k.shape[2])
    x = x.masked_fill(~seen, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    stored = (key < (ctx + (cu[1:] - cu[:-1]))[:, None])[:, None, :, None]
    o = torch.matmul(p, v.masked_fill(~stored, 0.0)) / p.sum(-1, keepdim=True)
    return o.view(count, hk, hq // hk, max_q, a).permute(0, 3, 1, 2, 4).reshape(count, max_q, hq, a)


def _attention(s):
    d, n = s["decodes"], s["ctx"].shape[0]
    out = torch.empty_like(s["q"])
    if d:
        out[:d] = _attend(s, 0, d, 1, s["max_decode_kv"])[:, 0].to(out.dtype)
    if n > d:
        o = _attend(s, d, n - d, s["max_q"], s["max_kv"])
        cu = s["cu"][d:].long()
        t = torch.arange(d, out.shape[0], device="cuda")
        r = torch.searchsorted(cu, t, right=True) - 1
        out[d:] = o[r, t - cu[r]].to(out.dtype)
    return out


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_cb_gb300 as cb
        cache = (s["k"], s["v"], s["k_exps"], s["v_exps"])
        if op == "append":
            cb.cb_kv_append_fp8(s["k_new"], s["v_new"], s["slots"], *cache)
        elif op == "gather":
            cb.cb_kv_gather_fp8(s["slots"], *cache, s["k_out"], s["v_out"])
        elif op == "step":
            cb.cb_kv_append_paged_attention_fp8(s["k_new"], s["v_new"], s["slots"], s["q"], s["cu"], s["ctx"],
                                                s["tables"], *cache, s["out"], s["scale"], s["workspace"], s["max_q"],
                                                s["max_kv"], window=s["window"])
        else:
            cb.cb_paged_attention_fp8(s["q"], s["cu"], s["ctx"], s["tables"], *cache, s["out"], s["scale"],
                                      s["workspace"], s["max_q"], s["max_kv"], window=s["window"])
        out = s.get("out")
    else:
        if op in ("append", "step"):
            _write(s["k"], s["k_exps"], s["slots"], s["k_new"])
            _write(s["v"], s["v_exps"], s["slots"], s["v_new"])
        if op == "gather":
            _read(s["k"], s["k_exps"], s["slots"], s["k_out"])
            _read(s["v"], s["v_exps"], s["slots"], s["v_out"])
        out = _attention(s) if op in ("decode", "chunk", "step") else None
    if op == "gather":
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "append":
        return {"k": s["k"], "v": s["v"], "k_exps": s["k_exps"], "v_exps": s["v_exps"]}
    if op == "step":
        return {"out": out, "k": s["k"], "v": s["v"], "k_exps": s["k_exps"], "v_exps": s["v_exps"]}
    return {"out": out}


def work(case):
    hq, hk, a = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("append", "gather"):
        n = case["tokens"]
        moved = n - (-(-n // case["skip"]) if case["skip"] else 0)
        return {"bytes": 8 * n + moved * hk * 2 * (2 * a + a + 1), "flops": moved * hk * 2 * 2 * a}
    w = case["window"]
    keys = pairs = tokens = 0
    for q, c in _lengths(case):
        tokens += q
        keys += min(c + q, q + w - 1) if w else c + q
        pairs += sum(min(c + i + 1, w) if w else c + i + 1 for i in range(q))
    moved = keys * hk * 2 * (a + 1) + tokens * hq * a * 4
    if case["op"] == "step":
        moved += tokens * hk * 2 * (2 * a + a + 1)
    return {"bytes": moved, "flops": 4 * a * hq * pairs}


# ---------------------------------------------------------------- the same in 64 bits
def _two(e):
    """2^e in float64, from a table of exact values."""
    table = torch.tensor([2.0 ** k for k in range(-160, 161)], dtype=torch.float64, device=e.device)
    return table[e + 160]


def _grid(x):
    """float64 rows [..., A] -> (e4m3 values as float64, exponents), by the definition; rows are finite."""
    big = x.abs().amax(-1)
    e = torch.ceil(torch.log2(big.clamp(min=2.0 ** -140) / 448)).long().clamp(min=-126)
    # log2 may be off by a rounding next to a border: put right by comparing
    e = torch.where(big > 448 * _two(e), e + 1, e)
    e = torch.where((e > -126) & (big <= 448 * _two(e - 1)), e - 1, e)
    y = x * _two(-e)[..., None]
    size = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).long()
    size = torch.where(y.abs() >= _two(size + 1), size + 1, size)
    size = torch.where((size > -6) & (y.abs() < _two(size)), size - 1, size)
    step = _two(size - 3)
    return torch.round(y / step) * step, e


def _bytes_to_double(cache):
    """e4m3 bits -> float64 from the format: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    b = cache.view(torch.uint8).long()
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e > 0, (1 + m / 8) * _two(e - 7), m * 2.0 ** -9)
    return torch.where(b >> 7 == 1, -x, x)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gather":
        res = {}
        for name in ("k", "v"):
            out = s[name + "_out"].double()
            for t0 in range(0, out.shape[0], 8192):
                sl = s["slots"][t0:t0 + 8192]
                idx = torch.nonzero(sl >= 0)[:, 0]
                blk, off = sl[idx] // BS, sl[idx] % BS
                scale = _two(s[name + "_exps"][blk, :, off].long() - 127)
                out[t0 + idx] = _bytes_to_double(s[name].view(torch.uint8)[blk, :, off]) * scale[..., None]
            res[name] = out
        return res
    caches = {}
    if op in ("append", "step"):
        if s["k"].numel() * 8 > 24 << 30:
            return None
        for name in ("k", "v"):
            full, exps = _bytes_to_double(s[name]), s[name + "_exps"].long() - 127
            for t0 in range(0, s["slots"].shape[0], 8192):
                y, e = _grid(s[name + "_new"][t0:t0 + 8192].double())
                sl = s["slots"][t0:t0 + 8192]
                idx = torch.nonzero(sl >= 0)[:, 0]
                full[sl[idx] // BS, :, sl[idx] % BS] = y[idx]
                exps[sl[idx] // BS, :, sl[idx] % BS] = e[idx]
            caches[name] = (full, exps)
        written = {"k": caches["k"][0], "v": caches["v"][0], "k_exps": None, "v_exps": None}
        if op == "append":
            return written
    if work(case)["flops"] > 1.2e13:
        return None
    reqs = _lengths(case)
    hq, hk, a = case["heads"], case["kv_heads"], case["dim"]
    g, out, t = hq // hk, torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for r, (q, c) in enumerate(reqs):
        n = c + q
        blk = s["tables"][r, :-(-n // BS)].long()
        kv = []
        for name in ("k", "v"):
            if op == "step":
                x, e = caches[name][0][blk], caches[name][1][blk]
            else:
                x, e = _bytes_to_double(s[name].view(torch.uint8)[blk]), s[name + "_exps"][blk].long() - 127
            x = x * _two(e)[..., None]
            kv.append(x.transpose(0, 1).reshape(hk, -1, a)[:, :n])
        pos = c + torch.arange(q, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        hidden = key > pos
        if case["window"]:
            hidden = hidden | (pos - key >= case["window"])
        for h in range(hk):
            x = torch.einsum("qgd,nd->gqn", s["q"][t:t + q, h * g:(h + 1) * g].double(), kv[0][h]) / math.sqrt(a)
            p = torch.softmax(x.masked_fill_(hidden, -math.inf), -1)
            out[t:t + q, h * g:(h + 1) * g] = torch.einsum("gqn,nd->qgd", p, kv[1][h])
        t += q
    return {"out": out, **written} if op == "step" else {"out": out}
