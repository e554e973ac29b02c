"""The paged cache on the GPU at the edges of what its header allows: wrong counts, damaged
tables, the largest batches, wide tables, and the kernels that only large calls take."""
import numpy as np
import pytest
import torch

from oracle.paged_oracle import D, PAGE, full
from pagedhelpers import Pair, bf16, check_attention, f32, i32
from quantized_kv_attention_int4_b200 import paged

pytestmark = pytest.mark.gpu

M = 2 ** 31 - 1


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 104729 * int(k) for i, k in enumerate(key)) + 71)


# ------------------------------------------------------------------------------- tables
@pytest.mark.parametrize("batch,max_pages", [(9, 8), (120, 8), (120, 200), (1300, 8)])
def test_counts_whose_total_passes_31_bits_touch_nothing_else(batch, max_pages):
    """Refused counts of up to 2^31 - 1 beside valid ones, in one block, in a cluster and over
    several chunks: entries behind 2^31 - 1 rows are refused, the others get their own pages."""
    r = np.random.default_rng(batch + max_pages)
    pair = Pair(batch, max_pages, 5 * batch, 1)
    x, o = pair.c.index, pair.o
    for huge in ([0, 1, 2], [batch // 2], [batch - 1], [batch // 3, batch // 3 + 1, batch // 2, batch - 2]):
        n = r.integers(0, 300, batch)
        n[r.random(batch) < 0.2] = 0
        n[huge] = M
        n[3] = 200
        sl = r.permutation(batch)
        sl[5] = -1
        start, cu = pair.c.extend(i32(sl), i32(n))
        ostart, ocu = o.extend(sl, n)
        assert start.tolist() == ostart.tolist() and cu.tolist() == ocu.tolist()
        pair.same_index()
        owned = torch.cat([x.table[s, : -(-int(o.length[s]) // PAGE)] for s in range(batch)] + [x.free_pages[: int(x.n_free)]])
        assert sorted(owned.tolist()) == list(range(5 * batch))
        pair.c.release(i32(sl[::2]))
        o.release(sl[::2], len(sl[::2]))
        pair.same_index()
    code, detail, count = pair.c.status()
    assert count == len(o.errors) and (code, detail) in o.errors
    assert {paged.FL_DEV_TOO_LONG, paged.FL_DEV_COUNT} <= {c for c, _ in o.errors}


def test_rows_up_to_the_last_that_offsets_can_name():
    """The last entry's rows end at 2^31 - 1 exactly: granted; one row more: refused."""
    for last, granted in ((7, True), (8, False)):
        pair = Pair(3, 4, 12, 1)
        n = [M - 7, last, 0]                    # the first is too long for its request
        start, cu = pair.c.extend(None, i32(n))
        assert start.tolist() == [-1, 0 if granted else -1, 0]
        assert cu.tolist() == [0, M - 7, M, M]
        assert pair.c.index.length.tolist() == [0, last if granted else 0, 0]
        assert pair.c.index.n_free.item() == (11 if granted else 12)
        assert pair.c.status()[2] == (1 if granted else 2)


@pytest.mark.parametrize("slots,max_pages", [(20, 10), (120, 30), (1100, 6)])
def test_damaged_table_entries_are_given_to_no_one(slots, max_pages):
    """Release of tables with entries that are no pages: the others come back in order, the next
    requests get pages only.  In one block, in a cluster, and over several chunks."""
    r = np.random.default_rng(slots)
    pages = slots * max_pages // 2
    pair = Pair(slots, max_pages, pages, 1)
    x, o = pair.c.index, pair.o
    n = r.integers(0, 64 * max_pages // 2, slots)
    n[0], n[1] = 64 * max_pages // 2, 65
    pair.c.extend(None, i32(n))
    o.extend(None, n)
    hit = [s for s in range(slots) if s < 2 or r.random() < 0.1 and n[s] > 0]
    for i, s in enumerate(hit):
        j = int(r.integers(0, -(-n[s] // PAGE)))
        o.table[s, j] = x.table[s, j] = (-1, pages, -5, M)[i % 4]
    order = r.permutation(slots)
    order[3] = -1
    order[[5, 6]] = 0, 1                        # damaged rows among them, whatever the order
    for part in (order[: slots // 2], order[slots // 2:]):
        pair.c.release(i32(part))
        o.release(part, len(part))
        pair.same_index()
    n_free = int(x.n_free.item())
    assert n_free < pages
    code, detail, count = pair.c.status()
    assert count == len(o.errors) and (code, detail) in o.errors and paged.FL_DEV_PAGE_RANGE in {c for c, _ in o.errors}
    o.errors.clear()
    sl = [s for s in range(slots) if o.length[s] == 0]
    n = np.full(len(sl), 64)
    start, cu = pair.c.extend(i32(sl), i32(n))
    ostart, _ = o.extend(sl, n)
    assert start.tolist() == ostart.tolist()
    pair.same_index()
    got = [int(x.table[s, 0]) for s, b in zip(sl, ostart) if b >= 0]
    assert len(set(got)) == len(got) and min(got) >= 0 and max(got) < pages


def test_slot_map_of_the_last_rows_that_offsets_can_name():
    x = paged.PagedIndex.empty(2, 4, 8)
    paged.fl_paged_extend(x, None, i32([90, 100]), i32([0, 0]), i32([0, 0, 0]))
    pos = torch.full((M,), -7, dtype=torch.int32, device="cuda")
    paged.fl_paged_slot_map(x, None, i32([3, 40]), i32([M - 11, M - 9, M]), None, pos)
    assert pos[M - 14:].tolist() == [-7] * 3 + [3, 4] + list(range(40, 49))


# ------------------------------------------------------------------------------- append and read
def test_append_stops_at_offsets_that_descend():
    g = gen(2)
    pair = Pair(5, 4, 20, 2)
    sl, n = [3, 1, 0, 4, 2], [70, 65, 5, 100, 64]
    start, cu = pair.c.extend(i32(sl), i32(n))
    pair.o.extend(sl, n)
    k, v = bf16(g, 400, 2, D), bf16(g, 400, 2, D)
    bad = [0, 70, 135, 130, 230, 294]           # the third entry's offsets descend
    pair.c.append(0, i32(sl), start, i32(bad), k.cuda(), v.cuda())
    assert pair.c.status() == [paged.FL_DEV_COUNT, 2, 1]
    pair.o.append(sl[:2], [0, 0], bad[:3], f32(k), f32(v))
    pool = pair.c.pools[0]
    for s in (0, 4, 2):
        assert torch.isnan(pool.tail_k[s]).all() and torch.isnan(pool.tail_v[s]).all()
    assert not pool.rec[1].any() and not pool.rec[3:].any()     # the first two's blocks are in pages 0 and 2
    sl[2] = -1                                  # also where the entry is padded
    pair.c.append(0, i32(sl), start, i32(bad), k.cuda(), v.cuda())
    assert pair.c.status() == [paged.FL_DEV_COUNT, 2, 1] and torch.isnan(pool.tail_k[4]).all()
    sl[2] = 0
    pair.c.append(0, i32(sl), start, cu, k.cuda(), v.cuda())
    pair.o.append(sl, [0] * 5, np.cumsum([0] + n), f32(k), f32(v))
    pair.same_bytes()
    assert pair.c.status()[2] == 0


def test_offsets_that_name_the_same_rows_again_and_again():
    """8192 entries, every other one with all of 2^20 rows of 64 heads: 2^33 items, were they counted."""
    batch, heads, rows = 8192, 64, 1 << 20
    x = paged.PagedIndex.empty(1, 16384, 4)
    pool = paged.PagedPool.empty(x, heads)
    pool.rec.zero_(), pool.tail_k.zero_(), pool.tail_v.zero_()
    k = bf16(gen(3), rows // 64, 1, D).cuda().repeat(64, 1, 1).expand(rows, heads, D)
    cu = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = rows
    zeros = torch.zeros(batch, dtype=torch.int32, device="cuda")
    paged.fl_paged_append(x, pool, zeros, zeros, cu, k, k)
    # the first entry has its tail; its pages are none (table -1), and every other entry is skipped
    assert torch.equal(pool.tail_k[0], k[-64:].transpose(0, 1)) and torch.equal(pool.tail_v[0], pool.tail_k[0])
    assert not pool.rec.any()
    assert x.status.tolist()[2] == batch // 2 + 16383 * heads


# ------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (1, 7)])
def test_tokens_of_infinitely_low_scores_have_no_weight(kv, group):
    """Blocks whose zero is -inf (keys below the 16-bit numbers) and tail rows of -inf: wherever
    they stand, first in a request or in a warp's part, the others' softmax is as without them."""
    g = gen(5, kv, group)
    lengths = [64 * 30 + 5, 65, 130, 84, 64 * 4 + 17, 1, 64 * 3 + 2, 33]
    pair = Pair(len(lengths), 32, 60, kv, kv * group)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    k, v = bf16(g, int(cu[-1]), kv, D), bf16(g, int(cu[-1]), kv, D)
    low = -66048.0 - 512.0 * (torch.arange(64) % 8)
    for b, n in enumerate(lengths):
        for j in range(full(n)):
            if b in (1, 6) or j % 2 == 0:
                k[cu[b] + 64 * j: cu[b] + 64 * j + 64, :, 0] = low[:, None].bfloat16()
    for b, rows in ((3, range(64, 80)), (4, range(256, 272)), (5, [0]), (6, [192, 193]), (7, range(0, 32))):
        k[[int(cu[b]) + t for t in rows], :, 0] = float("-inf")
    start, c = pair.c.extend(None, i32(lengths))
    pair.c.append(0, None, start, c, k.cuda(), v.cuda())
    s, oc = pair.o.extend(None, lengths)
    with np.errstate(over="ignore"):
        pair.o.append(None, s, oc, f32(k), f32(v))
    pair.same_bytes()
    q = bf16(g, len(lengths), kv * group, D, scale=1.5)
    q[..., 0] = q[..., 0].abs() + 0.125
    o = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    pair.c.attend(0, None, q.cuda(), o, lse)
    for b in (5, 6):
        assert not o[b].any() and torch.isneginf(lse[b]).all()
    live = [b for b in range(len(lengths)) if b not in (5, 6)]
    check_attention(pair, live, q[live], o[live], lse[live])
    for b in live:
        for h in range(kv):
            _, want = pair.o.attend(b, h, q[b, h * group: (h + 1) * group].double().numpy())
            # scores of up to 2^6 in base 2, each a sum of 128 products: 132 half steps at most
            assert np.abs(lse[b, h * group: (h + 1) * group].cpu().numpy() - want).max() <= 132 * 2.0 ** -24 * 64
    assert pair.c.status()[2] == 0


# ------------------------------------------------------------------------------- the largest batches
@pytest.mark.parametrize("batch", [8183, 8184, paged.MAX_BATCH])
def test_the_largest_batches_do_what_their_parts_do(batch):
    """Every call on a whole batch of up to 8192 entries against the same calls on 128 entries at a time."""
    r = np.random.default_rng(batch)
    g = gen(4, batch)
    kv, heads = 2, 6
    n = r.integers(0, 260, batch)
    x = paged.PagedIndex.empty(batch, 5, int(sum(-(-n // PAGE))))
    sl = i32(r.permutation(batch))
    start, cu = (torch.empty(batch + e, dtype=torch.int32, device="cuda") for e in (0, 1))
    paged.fl_paged_extend(x, sl, i32(n), start, cu)
    assert not start.any() and cu.tolist() == np.cumsum([0, *n]).tolist() and x.n_free.item() == 0
    t = int(n.sum())
    k, v = (bf16(g, 4096, kv, D).cuda().repeat(-(-t // 4096), 1, 1)[:t] for _ in range(2))
    q = bf16(g, batch, heads, D, scale=1.5).cuda()
    pools = [paged.PagedPool.empty(x, kv) for _ in range(2)]
    for p in pools:
        p.rec.zero_(), p.tail_k.zero_(), p.tail_v.zero_()
    place, pos = (torch.full((2, t), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    sel = torch.full((2, batch, kv, 2), -7, dtype=torch.int32, device="cuda")
    o = torch.full((4, batch, heads, D), 7.0, device="cuda")
    ws = [paged.workspace(x, pools[0], b, heads) for b in (batch, 128)]
    for i, step in enumerate((batch, 128)):
        for b in range(0, batch, step):
            e = slice(b, min(b + step, batch))
            at = cu[e.start: e.stop + 1].contiguous()
            paged.fl_paged_append(x, pools[i], sl[e], start[e], at, k, v)
            paged.fl_paged_slot_map(x, sl[e], start[e], at, place[i], pos[i])
            paged.fl_paged_select(x, pools[i], sl[e], q[e], sel[i, e], ws[i])
            paged.fl_paged_attn_decode(x, pools[i], sl[e], q[e], o[i, e], ws[i])
            paged.fl_paged_attn_decode(x, pools[i], sl[e], q[e], o[2 + i, e], ws[i], sel=sel[i, e])
    for name in ("rec", "tail_k", "tail_v"):
        assert torch.equal(getattr(pools[0], name), getattr(pools[1], name)), name
    assert torch.equal(place[0], place[1]) and torch.equal(pos[0], pos[1]) and not (place == -7).any()
    assert torch.equal(sel[0], sel[1]) and (sel >= -1).all()
    for i in (0, 2):
        # each side within check_attention's 4e-6 of the exact output, whatever the cuts between warps
        assert ((o[i] - o[i + 1]).norm(dim=-1) <= 8e-6 * o[i].norm(dim=-1)).all()
    assert x.status.tolist()[2] == 0
    paged.fl_paged_release(x, sl)
    assert not x.length.any() and sorted(x.free_pages.tolist()) == list(range(x.pages))
