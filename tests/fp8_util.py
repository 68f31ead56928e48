"""Helpers of the 8-bit cache tests: seeded steps over a quantised pool, the
fp64 oracle's view of them, and the elementwise error bound."""
import math

import numpy as np
import torch

from gpu_util import L, cu_of
from oracle import attention as oa
from oracle import fp8 as of8

BS = 16


class Step:
    """A ragged step over a random 8-bit pool.  ``reqs``: (q_len, ctx) pairs.
    Every slot that no request reads holds NaN patterns and odd exponents."""

    def __init__(self, reqs, hq, hk, a, seed=0, window=0, qscale=1.0, vspread=1, spare=3, kexp=(120, 123)):
        rng = np.random.default_rng(seed)
        self.reqs, self.hq, self.hk, self.a, self.window = list(reqs), hq, hk, a, window
        self.q_lens = [q for q, _ in reqs]
        self.ctx = [c for _, c in reqs]
        need = [-(-(q + c) // BS) if q else 0 for q, c in reqs]
        self.nb = sum(need) + spare
        order = rng.permutation(self.nb).astype(np.int32)
        self.tables = np.full((len(reqs), max(max(need, default=1), 1)), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.tables[r, :n] = order[at:at + n]
            at += n
        # rows like quantised normal ones: codes of N(0, 1) * 2^6, exponents near 2^-6
        shape = (self.nb, hk, BS, a)
        y = rng.standard_normal((2,) + shape) * 100
        mags = np.searchsorted(of8.VALUES, np.minimum(np.abs(y), 448))
        codes = (np.minimum(mags, 126) | np.where(y < 0, 128, 0)).astype(np.uint8)
        self.k_codes, self.v_codes = codes
        self.k_exps = rng.integers(kexp[0], kexp[1], shape[:3]).astype(np.uint8)
        self.v_exps = rng.integers(122 - vspread, 122 + vspread, shape[:3]).astype(np.uint8)
        used = np.zeros((self.nb, BS), bool)
        for r, (q, c) in enumerate(reqs):
            lo = max(0, c - window + 1) if window else 0
            for p in range(lo, q + c if q else 0):
                used[self.tables[r, p // BS], p % BS] = True
        stale = ~used[:, None, :] & np.ones((1, hk, 1), bool)
        for codes in (self.k_codes, self.v_codes):
            codes[stale] = rng.choice([0x7F, 0xFF], (int(stale.sum()), a))
        for exps in (self.k_exps, self.v_exps):
            exps[stale] = rng.choice([0, 1, 254, 255], int(stale.sum()))
        if window:      # blocks that left every window: released
            for r, (q, c) in enumerate(reqs):
                self.tables[r, :max(0, c - window + 1) // BS] = -1
        n = sum(self.q_lens)
        q = torch.from_numpy(rng.standard_normal((n, hq, a)) * qscale).to(torch.bfloat16)
        self.q = q
        self.scale = 1.0 / math.sqrt(a)

    # ------------------------------------------------------------ device side
    def cache(self, dev="cuda"):
        f = lambda x: torch.from_numpy(x.copy()).to(dev)  # noqa: E731
        return (f(self.k_codes).view(torch.float8_e4m3fn), f(self.v_codes).view(torch.float8_e4m3fn),
                f(self.k_exps), f(self.v_exps))

    @property
    def max_q(self):
        return max(max(self.q_lens), 1)

    @property
    def max_kv(self):
        return max(q + c for q, c in self.reqs)

    def workspace(self, dev="cuda", fill=None):
        n = L().cb_paged_attention_fp8_workspace_size(len(self.reqs), self.q.shape[0], self.max_q, self.max_kv, self.hq,
                                                      self.hk, self.a, BS)
        assert n > 0
        return torch.empty(n, dtype=torch.uint8, device=dev).fill_(0xFF if fill is None else fill)

    def meta(self, dev="cuda"):
        return (self.q.to(dev), torch.from_numpy(cu_of(self.q_lens)).to(dev),
                torch.tensor(self.ctx, dtype=torch.int32, device=dev), torch.from_numpy(self.tables).to(dev))

    def run(self, cache=None, workspace=None, out=None, meta=None, status=0, stream=None):
        lib = L()
        meta = meta or self.meta()
        cache = cache or self.cache()
        out = torch.full_like(meta[0], float("nan")) if out is None else out
        ws = self.workspace() if workspace is None else workspace
        lib.cb_paged_attention_fp8(*meta, *cache, out, self.scale, ws, self.max_q, self.max_kv, window=self.window,
                                   stream=stream)
        got = lib.cb_last_error(stream)
        assert got == status, lib.cb_strerror(got)
        return out

    # ------------------------------------------------------------ oracle
    def rows(self, r):
        """(K, V) of request r's keys in fp64, zeros before its window."""
        q, c = self.reqs[r]
        kv = []
        for codes, exps in ((self.k_codes, self.k_exps), (self.v_codes, self.v_exps)):
            out = np.zeros((q + c, self.hk, self.a))
            lo = max(0, c - self.window + 1) if self.window else 0
            p = np.arange(lo, q + c)
            blk = self.tables[r, p // BS]
            out[lo:] = of8.values(codes[blk, :, p % BS], exps[blk, :, p % BS])
            kv.append(out)
        return kv

    def reference(self):
        """(out, sum_j p_j |v_j|) of the step in fp64."""
        q = self.q.double().numpy()
        ks, vs = zip(*[self.rows(r) if self.q_lens[r] else [np.zeros((self.ctx[r], self.hk, self.a))] * 2
                       for r in range(len(self.reqs))])
        f = lambda v: oa.attention_step(q, self.q_lens, self.ctx, ks, v, self.scale, self.hq, self.hk,  # noqa: E731
                                        window=self.window)
        return f(vs), f([np.abs(v) for v in vs])


def check(got, ref, mag, what=""):
    """|got - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) sum_j p_j |v_j| elementwise:
    2^-8 |ref| is the output's rounding to bf16; each weight p_j carries one
    rounding to at least bf16 (2^-8); and its exponent's error, of the fp32 dot
    product (a sum of up to 128 products: 128 * 2^-24 of the sum of the products'
    magnitudes, at most some tens times log2 e here, so under 2^-11) and of
    2^x (2^-22), with the fp32 sums of p and p v (some hundred terms in a chain:
    2^-16), stays under 2^-10."""
    got = got.detach().double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mag
    worst = (np.abs(got - ref) / np.maximum(bound, 1e-300)).max() if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"
    return worst
