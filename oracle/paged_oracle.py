"""NumPy oracle of the paged cache of many requests (include/flashloop_paged.h): tables,
lengths and free pages request by request, records through the group codec of
flashloop_oracle, attention and scores in fp64.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

from . import flashloop_oracle as fo

PAGE, D, REC = 64, 128, 9216
SLOT_RANGE, SLOT_TWICE, NO_PAGE, TOO_LONG, COUNT, PAGE_RANGE = 16, 17, 18, 19, 20, 21


def full(n: int) -> int:
    """Blocks of a request of n tokens that are records (the last 1..64 tokens are not)."""
    return (n - 1) // PAGE if n > 0 else 0


def blocks(n: int) -> int:
    return -(-n // PAGE)


def record(k, v) -> np.ndarray:
    """The 9216 bytes of one block: k, v fp32 [64][128]."""
    e = fo.encode_base(k[None], v[None])
    out = np.zeros(REC, np.uint8)
    rows = out[: PAGE * D].reshape(PAGE, 2, D // 2)
    for i, c in enumerate((e["kc"][0], e["vc"][0])):
        rows[:, i] = c[:, 0::2] | (c[:, 1::2] << 4)
    out[8192:8704] = np.stack([e["vs"][0], e["vz"][0]], -1).reshape(-1).view(np.uint8)
    out[8704:] = np.stack([e["ks"][0, 0], e["kz"][0, 0]], -1).reshape(-1).view(np.uint8)
    return out


def unrecord(rec):
    """(k, v) fp64 [64][128] of one record, unrounded, and its key (scale, zero) [128][2]."""
    rows = rec[: PAGE * D].reshape(PAGE, 2, D // 2)
    c = np.empty((2, PAGE, D))
    for i in range(2):
        c[i, :, 0::2] = rows[:, i] & 15
        c[i, :, 1::2] = rows[:, i] >> 4
    vsz = rec[8192:8704].copy().view(np.float16).astype(np.float64).reshape(PAGE, 2, 2)
    ksz = rec[8704:].copy().view(np.float16).astype(np.float64).reshape(D, 2)
    return (c[0] * ksz[:, 0] + ksz[:, 1], c[1] * np.repeat(vsz[..., 0], D // 2, 1) + np.repeat(vsz[..., 1], D // 2, 1),
            ksz)


class PagedOracle:
    """One index and one pool; tails fp32 [slots][kv][64][128] holding BF16 values."""

    def __init__(self, slots, max_pages, pages, kv):
        self.table = np.full((slots, max_pages), -1, np.int64)
        self.length = np.zeros(slots, np.int64)
        self.free = list(range(pages - 1, -1, -1))
        self.rec = np.zeros((pages, kv, REC), np.uint8)
        self.tail = np.zeros((2, slots, kv, PAGE, D), np.float32)
        self.slots, self.max_pages, self.pages, self.kv = slots, max_pages, pages, kv
        self.errors = []

    def _named(self, slots, b, seen):
        s = b if slots is None else int(slots[b])
        if s == -1:
            return -1
        if not 0 <= s < self.slots:
            self.errors.append((SLOT_RANGE, b))
            return -1
        if s in seen:
            self.errors.append((SLOT_TWICE, b))
            return -1
        seen.add(s)
        return s

    def extend(self, slots, n_new):
        start, cu, seen, wanted, n_free = [], [0], set(), 0, len(self.free)
        for b, n in enumerate(int(n) for n in n_new):
            rows = cu[-1] + max(n, 0)
            cu.append(min(rows, 2 ** 31 - 1))
            s = self._named(slots, b, seen)
            start.append(-1)
            if s < 0:
                continue
            c = int(self.length[s])
            if n < 0:
                self.errors.append((COUNT, b))
                continue
            if c + n > self.max_pages * PAGE:
                self.errors.append((TOO_LONG, b))
                continue
            if n and rows > 2 ** 31 - 1:
                self.errors.append((COUNT, b))
                continue
            need = blocks(c + n) - blocks(c)
            wanted += need
            if need and wanted > n_free:
                self.errors.append((NO_PAGE, b))
                continue
            for j in range(blocks(c), blocks(c + n)):
                self.table[s, j] = self.free.pop()
            self.length[s] = c + n
            start[-1] = c
        return np.array(start), np.array(cu)

    def release(self, slots, batch):
        seen = set()
        for b in range(batch):
            s = self._named(slots, b, seen)
            if s < 0:
                continue
            for j in range(blocks(int(self.length[s]))):
                p = int(self.table[s, j])
                if 0 <= p < self.pages:
                    self.free.append(p)
                else:
                    self.errors.append((PAGE_RANGE, b))
                self.table[s, j] = -1
            self.length[s] = 0

    def place(self, s, t):
        return int(self.table[s, t // PAGE]) * PAGE + t % PAGE if t // PAGE < full(int(self.length[s])) \
            else (self.pages + s) * PAGE + t % PAGE

    def slot_map(self, slots, start, cu, n_tokens):
        place, pos = np.full(n_tokens, -7), np.full(n_tokens, -7)
        for b in range(len(start)):
            s = b if slots is None else int(slots[b])
            if not -1 <= s < self.slots and cu[b] < min(cu[b + 1], n_tokens):
                self.errors.append((SLOT_RANGE, b))
            for t in range(cu[b], min(cu[b + 1], n_tokens)):
                if not 0 <= s < self.slots or start[b] < 0:
                    place[t] = pos[t] = -1
                else:
                    pos[t] = start[b] + t - cu[b]
                    place[t] = self.place(s, int(pos[t])) if pos[t] < self.length[s] else -1
        return place, pos

    def append(self, slots, start, cu, k, v):
        """k, v fp32 [n_tokens][kv][128]."""
        for b in range(len(start)):
            s = b if slots is None else int(slots[b])
            n = int(cu[b + 1] - cu[b])
            if s < 0 or start[b] < 0 or n == 0:
                continue
            c = int(start[b])
            f0, f1 = full(c), full(c + n)
            for h in range(self.kv):
                rows = [np.concatenate([self.tail[i, s, h, : c - PAGE * f0], x[cu[b]: cu[b + 1], h]])
                        for i, x in enumerate((k, v))]
                for j in range(f0, f1):
                    cut = slice(PAGE * (j - f0), PAGE * (j - f0 + 1))
                    self.rec[self.table[s, j], h] = record(rows[0][cut], rows[1][cut])
                for i in range(2):
                    if f1 > f0:
                        last = rows[i][PAGE * (f1 - f0):]
                        self.tail[i, s, h, : len(last)] = last
                    else:
                        self.tail[i, s, h, c - PAGE * f0: c + n - PAGE * f0] = rows[i][c - PAGE * f0:]

    def keys_values(self, s, h, chosen=None):
        """fp64 K, V [n][128] of one request and head (of the chosen blocks and the tail)."""
        n = int(self.length[s])
        f = full(n)
        ks, vs = [np.zeros((0, D))], [np.zeros((0, D))]
        for j in range(f) if chosen is None else chosen:
            k, v, _ = unrecord(self.rec[self.table[s, j], h])
            ks.append(k)
            vs.append(v)
        ks.append(self.tail[0, s, h, : n - PAGE * f].astype(np.float64))
        vs.append(self.tail[1, s, h, : n - PAGE * f].astype(np.float64))
        return np.concatenate(ks), np.concatenate(vs)

    def select(self, s, h, q, keep):
        """Blocks of the highest score of one request and head, ascending: q fp64 [group][128]."""
        f = full(int(self.length[s]))
        if f <= keep:
            return list(range(f))
        scores = []
        for j in range(f):
            sz = unrecord(self.rec[self.table[s, j], h])[2]
            lo, hi = sz[:, 1], sz[:, 1] + 15 * sz[:, 0]
            scores.append(np.maximum(q * lo, q * hi).sum(-1).max())
        return sorted(sorted(range(f), key=lambda j: (-scores[j], j))[:keep])

    def attend(self, s, h, q, chosen=None):
        """(o [group][128], lse [group] in base 2) in fp64 of one request and head."""
        k, v = self.keys_values(s, h, chosen)
        if len(k) == 0:
            return np.zeros_like(q), np.full(len(q), -np.inf)
        x = q @ k.T / np.sqrt(D)
        m = x.max(-1, keepdims=True)
        p = np.exp(x - m)
        return p @ v / p.sum(-1, keepdims=True), (m[:, 0] + np.log(p.sum(-1))) / np.log(2.0)
