"""Definitions of the key-set operators in float64, and inputs for their tests.

`ref_attend` and `ref_mass` also return the bounds their results' rounding
errors obey, from the sizes of the operands:
  e_s   score error: a sum of D products in fp32 is off by at most
        D 2^-24 sum |q_i k_i| (times the scale), and scaling it rounds once more
  o     each output is sum_n p_n v_n / sum_n p_n: weights off by a factor
        exp(+-e_s) and by the exponential's own error (2^-22), bf16 weights by
        half a step (2^-8), the sums over N keys by N 2^-24 at most, and the
        stored value by half a step of its type
  lse   e_s, plus N 2^-24 of the sum, plus a few roundings of the value itself
  mass  each weight off by a factor exp(+-(e_s + the rounding of lse)), their
        sum over n terms by n 2^-24 at most
"""
import math

import numpy as np
import torch

U32 = 2.0 ** -24          # half a step of fp32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class Case:
    """One call's operands.  counts / lens: query rows and keys per sequence;
    listed: a random ascending list instead of the first lens[b] entries."""

    def __init__(self, dev, dtype, counts, lens, n_ctx, H, Hk, dh, prefix=0, listed=False,
                 seed=0, scale=0.0, pad=0, extra_rows=0, spread=1.0):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.dev, self.dt = dev, {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.dtype, self.counts, self.lens = dtype, list(counts), list(lens)
        self.B, self.n_ctx, self.H, self.Hk, self.dh = len(counts), n_ctx, H, Hk, dh
        self.prefix, self.scale = prefix, scale
        self.rows = sum(counts) + extra_rows

        def mat(n, cols, s=1.0):
            # row stride cols + pad; the padding holds NaN
            t = torch.full((max(n, 1), cols + pad), float("nan"), device=dev, dtype=self.dt)
            t[:, :cols] = (torch.randn((max(n, 1), cols), device=dev, generator=g) * s).to(self.dt)
            return t[:n, :cols]

        self.q = mat(self.rows, H * dh, spread)
        self.k, self.v = mat(self.B * n_ctx, Hk * dh), mat(self.B * n_ctx, Hk * dh)
        self.kp = mat(prefix, Hk * dh) if prefix else None
        self.vp = mat(prefix, Hk * dh) if prefix else None
        off = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        self.off = off
        self.seq_off = torch.from_numpy(off).to(dev)
        self.key_len = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.keys = None
        self.pos = [np.arange(n) for n in self.lens]
        if listed:
            rng = np.random.default_rng(seed)
            self.pos = [np.sort(rng.permutation(n_ctx)[:n]) for n in self.lens]
            tab = np.full((self.B, n_ctx), 1 << 30, dtype=np.int32)   # never to be read
            for b, p in enumerate(self.pos):
                tab[b, :len(p)] = p
            self.keys = torch.from_numpy(tab).to(dev)

    def key_attention(self, **kw):
        from token_locking_b200 import runtime as rt
        return rt.KeyAttention(self.B, self.n_ctx, max(self.rows, 1), self.H, self.dh, self.Hk,
                               self.dtype, prefix=self.prefix > 0, scale=self.scale, **kw)

    def poison(self, value=float("nan")):
        """Every cache row outside the key sets gets `value`."""
        live = torch.zeros(self.B * self.n_ctx, dtype=torch.bool, device=self.dev)
        for b, p in enumerate(self.pos):
            live[torch.from_numpy(np.asarray(p, dtype=np.int64)).to(self.dev) + b * self.n_ctx] = True
        self.k[~live] = value
        self.v[~live] = value
        return self

    def outputs(self, fill=7.0):
        o = torch.full((self.rows, self.H * self.dh), fill, dtype=self.dt, device=self.dev)
        return o, torch.full((self.rows, self.H), fill, device=self.dev)

    def attend(self, ka, o, lse, **kw):
        ka.attend(self.q, self.k, self.v, o, self.seq_off, key_len=self.key_len, keys=self.keys,
                  k_prefix=self.kp, v_prefix=self.vp, lse=lse, **kw)

    def _scores(self, b, h, with_prefix):
        r = slice(int(self.off[b]), int(self.off[b + 1]))
        hk = h * self.Hk // self.H
        col = slice(hk * self.dh, (hk + 1) * self.dh)
        idx = torch.from_numpy(np.asarray(self.pos[b], dtype=np.int64)).to(self.dev) + b * self.n_ctx
        q = self.q[r, h * self.dh:(h + 1) * self.dh].double()
        k, v = self.k[idx, col].double(), self.v[idx, col].double()
        if with_prefix and self.prefix:
            k = torch.cat([self.kp[:, col].double(), k])
            v = torch.cat([self.vp[:, col].double(), v])
        sc = self.scale if self.scale > 0 else 1.0 / math.sqrt(self.dh)
        z = q @ k.T * sc
        e = (q.abs() @ k.abs().T) * sc * (self.dh + 2) * U32
        return r, z, e, v


def ref_attend(c):
    """(o, o bound, lse, lse bound) in float64; untouched rows are NaN."""
    o = torch.full((c.rows, c.H, c.dh), float("nan"), dtype=torch.float64, device=c.dev)
    lse = torch.full((c.rows, c.H), float("nan"), dtype=torch.float64, device=c.dev)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(c.B):
        for h in range(c.H):
            r, z, e, v = c._scores(b, h, True)
            if z.shape[0] == 0:
                continue
            if z.shape[1] == 0:
                o[r, h], lse[r, h] = 0.0, -math.inf
                continue
            n = z.shape[1]
            ls = torch.logsumexp(z, dim=1)
            p = torch.exp(z - ls[:, None])
            o[r, h], lse[r, h] = p @ v, ls
            es = e.amax(dim=1, keepdim=True)
            # a running maximum may lag by 2^8, so a weight's exponent is rounded near 20
            rel = 2 * es + 2.0 ** -20 + n * U32
            if c.dt == torch.bfloat16:
                rel = rel + HALF[c.dt]
            a = p @ v.abs()
            bo[r, h] = 1.01 * (rel * a + HALF[c.dt] * (o[r, h].abs() + rel * a)) + 1e-30
            bl[r, h] = es[:, 0] + n * U32 + 8 * U32 * (ls.abs() + 16.0)
    return o.reshape(c.rows, c.H * c.dh), bo.reshape(c.rows, c.H * c.dh), lse, bl


def ref_mass(c, lse, prev=None, decay=0.0):
    """(mass, bound) in float64 from the given fp32 lse."""
    m = torch.zeros((c.B, c.n_ctx), dtype=torch.float64, device=c.dev)
    bound = torch.zeros_like(m)
    for b in range(c.B):
        pos = torch.from_numpy(np.asarray(c.pos[b], dtype=np.int64)).to(c.dev)
        n = c.counts[b] * c.H
        for h in range(c.H):
            r, z, e, _ = c._scores(b, h, False)
            if z.numel() == 0:
                continue
            ls = lse[r, h:h + 1].double()
            w = torch.where(torch.isinf(ls) & (ls < 0), torch.zeros_like(z), torch.exp(z - ls))
            # lse and score in base 2, each rounded once or twice, and the exponential's error
            es = e + 8 * U32 * (z.abs() + ls.abs().clamp(max=1e4)) + 2.0 ** -20
            m[b].index_add_(0, pos, w.sum(dim=0))
            bound[b].index_add_(0, pos, (w * 1.01 * (es + n * U32)).sum(dim=0))
    if prev is not None and decay != 0.0:
        m += decay * prev.double()
        bound += 4 * U32 * (decay * prev.double()).abs()
    return m, bound + 4 * U32 * m.abs() + 1e-30


def ref_evict(mass, budget, protect=None, present=None):
    """Per sequence the kept positions, from sorting."""
    B, N = mass.shape
    out = []
    for b in range(B):
        here = [i for i in range(N) if present is None or present[b, i]]
        fixed = [i for i in here if protect is not None and protect[b, i]]
        cand = [i for i in here if protect is None or not protect[b, i]]
        val = {i: (-math.inf if math.isnan(mass[b, i]) else float(mass[b, i])) for i in cand}
        cand.sort(key=lambda i: (-val[i], i))
        out.append(sorted(fixed + cand[:max(0, budget - len(fixed))]))
    return out
