"""Cases and float64 references of the 16-bit K/V layers (tests only)."""
import math

import numpy as np
import torch

BLOCK = 128
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
ST_BAD_POSITION, ST_BAD_INDEX, ST_BAD_SEQ = 1, 2, 4


class Case:
    """A ragged batch over a shuffled pool.  Every pool row that no position
    below kv_len maps to, and every spare block, holds NaN."""

    def __init__(self, ns, ls, Hq, Hkv, d, dtype="bf16", seed=0, q_scale=1.5, spare=3, bps=None,
                 front=0, behind=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.ns, self.ls, self.Hq, self.Hkv, self.d, self.dt = ns, ls, Hq, Hkv, d, DT[dtype]
        self.B, self.device = len(ns), device
        need = [-(-x // BLOCK) for x in ls]
        self.bps = bps or max(need + [1])
        self.n_blocks = sum(need) + spare
        ids = torch.randperm(self.n_blocks, generator=g)[:sum(need)].tolist()
        table = np.full((self.B, self.bps), -1, np.int32)
        for b, m in enumerate(need):
            table[b, :m], ids = ids[:m], ids[m:]
        self.table = table
        # token rows in front of the first and behind the last sequence belong to none
        self.start = np.cumsum([front] + list(ns)).astype(np.int32)
        self.T = int(self.start[-1]) + behind
        self.hist_k = [torch.randn(x, Hkv, d, generator=g).to(self.dt) for x in ls]
        self.hist_v = [torch.randn(x, Hkv, d, generator=g).to(self.dt) for x in ls]
        self.q = (q_scale * torch.randn(self.T, Hq, d, generator=g)).to(self.dt)
        pools = []
        for hist in (self.hist_k, self.hist_v):
            pool = torch.full((self.n_blocks, Hkv, BLOCK, d), math.nan, dtype=self.dt)
            for b, x in enumerate(ls):
                for i in range(0, x, BLOCK):
                    m = min(BLOCK, x - i)
                    pool[table[b, i // BLOCK], :, :m] = hist[b][i:i + m].transpose(0, 1)
            pools.append(pool)
        self.k_pool, self.v_pool = pools

    def tokens(self):
        """(token row, sequence, position) of every new token."""
        for b, (n, L) in enumerate(zip(self.ns, self.ls)):
            for i in range(n):
                yield int(self.start[b]) + i, b, L - n + i

    def args(self, ws):
        dev = self.device
        return dict(k_cache=self.k_pool.to(dev), v_cache=self.v_pool.to(dev),
                    q_start=torch.from_numpy(self.start).to(dev),
                    kv_len=torch.tensor(self.ls, dtype=torch.int64, device=dev),
                    block_table=torch.from_numpy(self.table).to(dev), ws=ws)


def counted(entries, last):
    """The blocks that a list's entries select for a query in block ``last``."""
    got, top = set(), -1
    for e in entries:
        if e >= 0 and e > top and e <= last:
            got.add(int(e))
        top = max(top, int(e))
    return got


def reference(c, n_win=0, sink=None, idx=None, n_local=0, scale=None, bad=()):
    """float64 (out, lse, tol_out, tol_lse) of every token row, NaN for rows
    that belong to no sequence.  ``bad``: (sequence, block) pairs not seen.

    Tolerances, with u the type's half step (2^-8 bf16, 2^-11 fp16):
    a softmax weight entering the product is off by u (its rounding) and by
    e_s (its score: fp32 dot products of d terms, at most d 2^-23 sum|q k|
    scale; exp2 2^-18), the sum of the weights by e_s, the result by u:
      |out - ref| <= u |ref| + (u + 2 e_s) sum_j w_j |v_j| (1 + u),
      |lse - ref| <= e_s + 2^-21 (1 + |lse|)."""
    u = torch.finfo(c.dt).eps / 2
    scale = scale or 1 / math.sqrt(c.d)
    g = c.Hq // c.Hkv
    out = torch.full((c.T, c.Hq, c.d), math.nan, dtype=torch.float64)
    lse = torch.full((c.T, c.Hq), math.nan, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for t, b, p in c.tokens():
        for h in range(c.Hkv):
            j = torch.arange(max(p + 1, 0))
            if n_win:
                j = j[j > p - n_win]
            if idx is not None:
                last = p // BLOCK
                sel = counted(idx[t, h if idx.shape[1] > 1 else 0].tolist(), last)
                sel |= set(range(max(0, last - n_local + 1), last + 1)) if n_local else set()
                j = j[[int(x) // BLOCK in sel for x in j]] if p >= 0 else j
            j = j[[(b, int(x) // BLOCK) not in bad for x in j]] if bad else j
            hs = slice(h * g, h * g + g)
            q = c.q[t, hs].double()
            k, v = c.hist_k[b][j, h].double(), c.hist_v[b][j, h].double()
            s = q @ k.T * scale
            e_s = c.d * 2.0 ** -23 * scale * (q.abs() @ k.abs().T)
            e_s = (e_s.amax(1) if len(j) else torch.zeros(g, dtype=torch.float64)) + 2.0 ** -18
            full = s if sink is None else torch.cat((s, sink[hs].double()[:, None]), 1)
            z = torch.logsumexp(full, 1) if full.shape[1] else torch.full((g,), -math.inf,
                                                                          dtype=torch.float64)
            w = (s - z[:, None]).exp() if len(j) else s
            out[t, hs], lse[t, hs] = w @ v, z
            tol_o[t, hs] = u * (w @ v).abs() + ((u + 2 * e_s)[:, None] * (w @ v.abs())) * (1 + u)
            tol_l[t, hs] = e_s + 2.0 ** -21 * (1 + torch.where(z.isfinite(), z.abs(), 0.0))
    return out, lse, tol_o, tol_l


def check(c, got_out, got_lse, ref, skip=()):
    """The kernel's rows against the reference; rows of no sequence must still
    hold the sentinel 7.0."""
    out, lse, tol_o, tol_l = ref
    o, z = got_out.double().cpu(), got_lse.double().cpu()
    mine = torch.zeros(c.T, dtype=torch.bool)
    for t, _, _ in c.tokens():
        mine[t] = True
    assert (o[~mine] == 7.0).all() and (z[~mine] == 7.0).all()
    for t in skip:
        mine[t] = False
    over = (o - out).abs()[mine] - tol_o[mine]
    assert o[mine].isfinite().all()
    assert (over <= 0).all(), f"out is off by {over.max():.3g} more than allowed"
    inf = lse[mine].isinf()
    assert torch.equal(z[mine].isinf(), inf) and (z[mine][inf] < 0).all()
    over = ((z - lse).abs() - tol_l)[mine][~inf]
    assert (over <= 0).all(), f"lse is off by {over.max():.3g} more than allowed"


def rotated(x, pos, d_rope, theta, halves):
    """float64 R(pos) on the last d_rope dims of x [T][H][d]."""
    x = x.double().clone()
    off = x.shape[-1] - d_rope
    for k in range(d_rope // 2):
        i = off + (k if halves else 2 * k)
        j = i + (d_rope // 2 if halves else 1)
        a = torch.as_tensor(pos, dtype=torch.float64) * theta ** (-2.0 * k / d_rope)
        cos, sin = a.cos()[:, None], a.sin()[:, None]
        x[..., i], x[..., j] = x[..., i] * cos - x[..., j] * sin, x[..., i] * sin + x[..., j] * cos
    return x
