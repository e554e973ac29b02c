"""Test-side helpers of the paged cache: a GPU cache and the oracle fed the same inputs."""
from __future__ import annotations

import numpy as np
import torch

from oracle.paged_oracle import D, PAGE, PagedOracle, full
from quantized_kv_attention_int4_b200.paged import PagedCache


def bf16(g, *shape, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g) * scale + shift).to(torch.bfloat16)


def f32(t):
    return t.float().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Pair:
    """A PagedCache of one plane and its oracle."""

    def __init__(self, slots, max_pages, pages, kv, q_heads=None, max_batch=None):
        self.c = PagedCache(1, kv, slots, max_pages * PAGE, pages, q_heads, max_batch)
        self.c.pools[0].rec.zero_()
        # rows that no token has reached hold NaN
        self.c.pools[0].tail_k.fill_(float("nan"))
        self.c.pools[0].tail_v.fill_(float("nan"))
        self.o = PagedOracle(slots, max_pages, pages, kv)
        self.o.tail[:] = np.nan
        self.kv = kv

    def step(self, slots, n_new, g, scale=1.0):
        """Extend and append seeded rows on both sides; returns (start, cu) of the GPU."""
        sl = None if slots is None else i32(slots)
        start, cu = self.c.extend(sl, i32(n_new))
        t = int(sum(max(n, 0) for n in n_new))
        chan = torch.exp(torch.randn(1, self.kv, D, generator=g) * 0.3)
        k = (bf16(g, max(t, 1), self.kv, D).float() * chan * scale + 0.5 * torch.randn(1, self.kv, D, generator=g)).bfloat16()
        v = bf16(g, max(t, 1), self.kv, D, scale=scale)
        self.c.append(0, sl, start, cu, k.cuda(), v.cuda())
        ostart, ocu = self.o.extend(slots, n_new)
        assert start.tolist() == ostart.tolist() and cu.tolist() == ocu.tolist()
        self.o.append(slots, ostart, ocu, f32(k), f32(v))
        return start, cu

    def same_index(self):
        x = self.c.index
        assert x.length.tolist() == self.o.length.tolist()
        n = int(x.n_free.item())
        assert n == len(self.o.free) and x.free_pages[:n].tolist() == self.o.free
        for s in range(self.o.slots):
            b = -(-int(self.o.length[s]) // PAGE)
            assert x.table[s, :b].tolist() == self.o.table[s, :b].tolist()

    def same_bytes(self):
        """Records and live tail rows equal byte for byte."""
        pool = self.c.pools[0]
        rec, tk, tv = pool.rec.cpu().numpy(), f32(pool.tail_k), f32(pool.tail_v)
        for s in range(self.o.slots):
            n = int(self.o.length[s])
            for j in range(full(n)):
                p = self.o.table[s, j]
                assert np.array_equal(rec[p], self.o.rec[p]), (s, j)
            r = n - PAGE * full(n)
            assert np.array_equal(tk[s, :, :r], self.o.tail[0, s, :, :r]), s
            assert np.array_equal(tv[s, :, :r], self.o.tail[1, s, :, :r]), s


def attention_tol(q, k, v, x_scale):
    """Worst-case rounding bound of one head's fp32 attention (absolute, on o and on lse).

    A score is a sum of 128 products and a few further operations: it is off by at most
    e = 132 u sum_c |q_c k_c| x_scale (u = 2^-24) plus 2 u of its own magnitude; a weight by
    ln2 e relatively, the exponential's 2^-22, the weight's own rounding to two 16-bit parts
    2^-22, and the rescaling of running sums (3 u a block of 64).  o is a quotient of two sums
    of n such weights, each summed with n u relative to the sum of magnitudes at most."""
    u = 2.0 ** -24
    n = len(k)
    if n == 0:
        return 0.0, 0.0
    mag = float((np.abs(q) @ np.abs(k).T).max()) * x_scale
    e = 132 * u * mag + 2 * u * mag
    rel = np.log(2.0) * e + 2 * 2.0 ** -22 + (3 * (n / 64 + 1) + n) * u
    return 2.5 * rel * float(np.abs(v).max()), 1.5 * rel / np.log(2.0) + 4 * u * (mag + np.log2(n + 1))


LOG2 = 1.4426950408889634 / np.sqrt(128.0)


def check_attention(pair, slots, q, o, lse, chosen=None):
    """o [batch][heads][128], lse [batch][heads] of the GPU against the oracle."""
    qn, on, ln = q.double().cpu().numpy(), o.cpu().numpy(), lse.cpu().numpy()
    kv = pair.kv
    group = qn.shape[1] // kv
    for b in range(len(qn)):
        s = b if slots is None else int(slots[b])
        for h in range(kv):
            hs = slice(h * group, (h + 1) * group)
            ch = None if chosen is None else chosen[b][h]
            ref, rl = pair.o.attend(s, h, qn[b, hs], ch)
            k, v = pair.o.keys_values(s, h, ch)
            to, tl = attention_tol(qn[b, hs], k, v, LOG2)
            err = np.abs(on[b, hs] - ref).max()
            assert err <= to, (b, s, h, err, to)
            if len(k) == 0:
                assert np.all(np.isneginf(ln[b, hs]))
                continue
            # beside the worst case: errors add up like noise, far below it
            assert np.linalg.norm(on[b, hs] - ref) <= 4e-6 * np.linalg.norm(ref), (b, s, h)
            assert np.abs(ln[b, hs] - rl).max() <= tl, (b, s, h)
