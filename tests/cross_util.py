"""Helpers of the cross attention tests: seeded batches over a paged cache, their
definition in float64 and the elementwise error bound."""
import math

import numpy as np
import torch

from gpu_util import L, cu_of

BS = 16


class Batch:
    """Requests (new tokens, stored keys) over a random pool.  Every slot that no
    request reads holds NaNs and infinities, table entries past a request's blocks
    hold junk."""

    def __init__(self, reqs, hq, hk, a, seed=0, qscale=1.0, kscale=1.0, extra_tokens=0, spare=3, num_blocks=None, first=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.reqs, self.hq, self.hk, self.a = list(reqs), hq, hk, a
        self.q_lens, self.kv = [q for q, _ in reqs], [n for _, n in reqs]
        need = [-(-n // BS) for n in self.kv]
        used_blocks = sum(need) + spare
        self.nb = num_blocks or used_blocks
        order = first + rng.permutation(used_blocks)
        self.width = max(max(need, default=1), 1) + 1
        self.tables = np.tile(np.array([-3, 1 << 30], np.int32), (len(reqs), self.width))[:, :self.width]
        at = 0
        for r, n in enumerate(need):
            self.tables[r, :n] = order[at:at + n]
            at += n
        bad = torch.tensor([math.nan, math.inf, -math.inf], device="cuda", dtype=torch.bfloat16)
        self.k = torch.zeros(self.nb, hk, BS, a, device="cuda", dtype=torch.bfloat16)
        self.v = torch.zeros_like(self.k)
        for t, scale in ((self.k, kscale), (self.v, 1.0)):
            part = torch.randn(used_blocks, hk, BS, a, device="cuda", generator=g) * scale
            t[first:first + used_blocks] = part.to(torch.bfloat16)
            for blk in order[at:]:
                t[int(blk)] = bad[torch.randint(0, 3, (hk, BS, a), device="cuda", generator=g)]
            for r, n in enumerate(self.kv):
                if n % BS:
                    t[int(self.tables[r, n // BS]), :, n % BS:] = bad[torch.randint(0, 3, (hk, BS - n % BS, a), device="cuda",
                                                                                    generator=g)]
        n = sum(self.q_lens) + extra_tokens
        self.q = (torch.randn(n, hq, a, device="cuda", generator=g) * qscale).to(torch.bfloat16)
        self.scale = 1.0 / math.sqrt(a)
        self.d_cu = torch.from_numpy(cu_of(self.q_lens)).cuda()
        self.d_kv = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        self.d_tables = torch.from_numpy(np.ascontiguousarray(self.tables)).cuda()

    @property
    def max_q(self):
        return max(max(self.q_lens), 1)

    @property
    def max_kv(self):
        return max(self.kv)

    def workspace(self):
        n = L().cb_paged_cross_attention_workspace_size(len(self.reqs), self.q.shape[0], self.max_q, self.max_kv, self.hq,
                                                        self.hk, self.a, BS)
        assert n > 0
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, out=None, ws=None, check=True, stream=None):
        lib = L()
        out = torch.full_like(self.q, 7.0) if out is None else out
        ws = self.workspace() if ws is None else ws
        lib.cb_paged_cross_attention(self.q, self.d_cu, self.d_kv, self.d_tables, self.k, self.v, out, self.scale, ws,
                                     self.max_q, self.max_kv, stream=stream)
        if check:
            status = lib.cb_last_error(stream)
            assert status == 0, lib.cb_strerror(status)
        return out

    def request(self, r):
        """K and V of request r, float64 [Hkv, keys, A]."""
        n = self.kv[r]
        blk = torch.from_numpy(self.tables[r, :-(-n // BS)].astype(np.int64)).cuda()
        return [t[blk].transpose(0, 1).reshape(self.hk, -1, self.a)[:, :n].double() for t in (self.k, self.v)]

    def compare(self, out, requests=None):
        """Every element against the definition in float64.

        The bound: bf16 rounds the output and every weight by at most 2^-8 of itself.
        A score is a sum of A exact products in fp32 whose order is the hardware's:
        within A 2^-23 sum |q||k| scale = e; the argument of the exponential adds its
        own rounding, its factor's and ex2's, (1 + |score|) 2^-20 in all.  Both
        weights of a ratio may be off by that much; the fp32 sum over n keys adds
        n 2^-23."""
        g, t0 = self.hq // self.hk, 0
        for r, (q, n) in enumerate(self.reqs):
            got = out[t0:t0 + q].double()
            if q and not n:
                assert not got.any(), f"request {r}: no keys, not zero"
            elif q and (requests is None or r in requests):
                k, v = self.request(r)
                for h in range(self.hk):
                    x = self.q[t0:t0 + q, h * g:(h + 1) * g].double()
                    s = torch.einsum("qgd,nd->gqn", x, k[h]) * self.scale
                    p = torch.softmax(s, -1)
                    ref = torch.einsum("gqn,nd->qgd", p, v[h])
                    size = torch.einsum("gqn,nd->qgd", p, v[h].abs())
                    e = self.a * 2.0 ** -23 * self.scale * torch.einsum("qgd,nd->gqn", x.abs(), k[h].abs()).amax(-1)
                    e = e + (1 + s.abs().amax(-1)) * 2.0 ** -20
                    weight = 2.0 ** -8 + 2 * torch.expm1(e).transpose(0, 1)[..., None] + n * 2.0 ** -23
                    bound = (2.0 ** -8 * ref.abs() + weight * size) * (1 + 2.0 ** -8) + 2.0 ** -133
                    err = (got[:, h * g:(h + 1) * g] - ref).abs()
                    worst = float((err / bound).max())
                    assert worst <= 1, f"request {r} ({q} tokens, {n} keys), head group {h}: {worst:.2f} of the bound"
            t0 += q
        assert (out[t0:] == 7.0).all(), "rows behind the last request were written"
