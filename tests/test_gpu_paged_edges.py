"""The paged cache on the GPU at the edges of what its header allows: wrong counts, damaged
tables, the largest batches, wide tables, and the kernels that only large calls take."""
import numpy as np
import pytest
import torch

from oracle import flashloop_oracle as fo
from oracle.paged_oracle import D, PAGE, REC, full
from pagedhelpers import Pair, bf16, check_attention, f32, i32
from quantized_kv_attention_int4_b200 import abi, paged
from quantized_kv_attention_int4_b200.cache import FlashLoopCache

pytestmark = pytest.mark.gpu

M = 2 ** 31 - 1


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 104729 * int(k) for i, k in enumerate(key)) + 71)


def random_cache(lengths, max_pages, kv, group, seed, kinds=None):
    """A pair whose requests hold random records and tails (of `kinds` different key scales and
    zeros, if given): (pair, slots)."""
    r = np.random.default_rng(seed)
    pages = sum(-(-n // PAGE) for n in lengths) + 3
    pair = Pair(len(lengths) + 1, max_pages, pages, kv, kv * group, max_batch=len(lengths))
    slots = r.permutation(len(lengths) + 1)[: len(lengths)].tolist()
    start, _ = pair.c.extend(i32(slots), i32(lengths))
    ostart, _ = pair.o.extend(slots, lengths)
    assert start.tolist() == ostart.tolist() == [0] * len(lengths)
    rec = r.integers(0, 256, (pages, kv, REC), dtype=np.uint8)
    words = rec[..., 8192:].view(np.float16).reshape(pages, kv, 256, 2)     # 128 of values, 128 of channels
    words[..., 0] = 0.2 * np.exp(0.3 * r.standard_normal(words.shape[:3]))
    words[..., 1] = -7.5 * words[..., 0] + 0.3 * r.standard_normal(words.shape[:3])
    if kinds:
        words[:, :, 128:] = words[r.integers(0, kinds, pages), :, 128:]
    pair.o.rec[:] = rec
    tail = torch.from_numpy(r.standard_normal(pair.o.tail.shape).astype(np.float32)).bfloat16()
    pair.o.tail[:] = tail.float().numpy()
    pool = pair.c.pools[0]
    pool.rec.copy_(torch.from_numpy(rec))
    pool.tail_k.copy_(tail[0]), pool.tail_v.copy_(tail[1])
    return pair, slots


def best_blocks(pair, s, h, q, keep):
    """The selection by its definition in fp64, blocks that are not finite behind all others."""
    f = full(int(pair.o.length[s]))
    if f <= keep:
        return list(range(f))
    sz = pair.o.rec[pair.o.table[s, :f], h, 8704:].copy().view(np.float16).astype(np.float64).reshape(f, D, 2)
    lo, hi = sz[..., 1], sz[..., 1] + 15 * sz[..., 0]
    score = np.maximum(q[:, None] * lo, q[:, None] * hi).sum(-1).max(0)
    bad = ~np.isfinite(sz).all((1, 2))
    return sorted(sorted(range(f), key=lambda j: (bad[j], 0.0 if bad[j] else -score[j], j))[:keep])


def check_selection(pair, slots, q, sel, keep):
    """sel int32 [batch][kv][keep] of the GPU; returns the chosen blocks."""
    qn, got, chosen = q.double().numpy(), sel.cpu().numpy(), []
    group = q.shape[1] // pair.kv
    for b, s in enumerate(slots):
        chosen.append([best_blocks(pair, s, h, qn[b, h * group: (h + 1) * group], keep) for h in range(pair.kv)])
        for h, want in enumerate(chosen[-1]):
            assert got[b, h].tolist() == want + [-1] * (keep - len(want)), (b, h)
    return chosen


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


@pytest.mark.parametrize("batch,max_pages", [(100, 40), (700, 5)])
def test_captured_requests_that_leave_and_come(batch, max_pages):
    """Release, extend and slot map as clusters, captured once and replayed with other requests and counts."""
    r = np.random.default_rng(batch)
    pair = Pair(batch + 50, max_pages, batch * max_pages // 3, 1)
    x, o, t = pair.c.index, pair.o, 64 * batch
    gone, come, n = (torch.empty(b, dtype=torch.int32, device="cuda") for b in (batch // 2, batch, batch))
    start, cu = (torch.empty(batch + e, dtype=torch.int32, device="cuda") for e in (0, 1))
    place, pos = (torch.empty(t, dtype=torch.int32, device="cuda") for _ in range(2))
    gone.fill_(-1), come.fill_(-1), n.zero_()

    def step():
        paged.fl_paged_release(x, gone)
        paged.fl_paged_extend(x, come, n, start, cu)
        paged.fl_paged_slot_map(x, come, start, cu, place, pos)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(6):
        leave, enter = r.permutation(batch + 50)[: batch // 2], r.permutation(batch + 50)[:batch]
        leave[r.random(len(leave)) < 0.1] = -1
        new = r.integers(0, 128, batch)
        new[-1] = max(0, t - int(new[:-1].sum())) if i == 3 else new[-1]
        gone.copy_(i32(leave)), come.copy_(i32(enter)), n.copy_(i32(new))
        place.fill_(-7), pos.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        o.release(leave, len(leave))
        ostart, ocu = o.extend(enter, new)
        assert start.tolist() == ostart.tolist() and cu.tolist() == ocu.tolist()
        pair.same_index()
        oplace, opos = o.slot_map(enter, ostart, ocu, t)
        assert place.tolist() == oplace.tolist() and pos.tolist() == opos.tolist()
    code, detail, count = pair.c.status()
    assert count == len(o.errors) and (not count or (code, detail) in o.errors)


def test_a_cache_whose_every_call_is_on_another_stream():
    g = gen(14)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pair = Pair(4, 40, 120, 2, 8)
        for slots, n in (([2, 0, 3], [700, 1, 64 * 35]), ([0, 2, 1], [129, 1, 5]), ([3], [1])):
            pair.step(slots, n, g)
        q = bf16(g, 4, 8, D, scale=1.5)
        lse = torch.empty(4, 8, device="cuda")
        o = pair.c.attend(0, None, q.cuda(), lse=lse)
        sel = pair.c.select(0, None, q.cuda(), 6)
        place, _ = pair.c.places(i32([2]), i32([0]), i32([0, 701]), 701)
        k, v = pair.c.read(0, place)
        pair.same_bytes()
        check_attention(pair, None, q, o, lse)
        check_selection(pair, range(4), q, sel, 6)
        for got, ref in zip((k, v), pair.o.keys_values(2, 1)):
            assert torch.equal(got[:, 1].cpu(), torch.from_numpy(ref.astype(np.float32)).bfloat16())
        pair.c.release(None)
        assert pair.c.index.n_free.item() == 120 and pair.c.status()[2] == 0


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


@pytest.mark.parametrize("kv", [17, 33])
def test_append_of_more_than_16_heads(kv):
    """Requests that fill no block are one item per 16 heads: the last item has fewer."""
    g = gen(6, kv)
    pair = Pair(3, 3, 8, kv)
    for slots, n in (([0, 2, 1], [1, 64, 30]), ([2, 1], [1, 3]), ([0, 1], [63, 31]), (None, [1, 2, 3])):
        pair.step(slots, n, g)
        pair.same_bytes()
    assert pair.c.status()[2] == 0


def test_records_are_the_single_sequence_encoders_whatever_the_values():
    """NaN, infinities, numbers beyond and below the 16-bit ones and zeros of both signs, alone and
    mixed in a group: the same bytes as fl_encode_base (whose quantiser the header names)."""
    r = np.random.default_rng(17)
    heads, n = 2, 64 * 40
    odd = np.array([np.nan, np.inf, -np.inf, 7e4, -7e4, 3e38, -3e38, 1e-40, -1e-40, 0.0, -0.0, 65504.0, 65520.0, -65535.0])
    kv = []
    for _ in range(2):
        x = r.standard_normal((heads, n, D)) * np.exp2(r.integers(-20, 16, (heads, n // 64, D)).repeat(64, 1))
        x = np.where(r.random(x.shape) < r.choice([0.0, 0.01, 0.3], (heads, n // 64, D)).repeat(64, 1), r.choice(odd, x.shape), x)
        x[0, :64, :14] = odd                    # whole groups of one value
        kv.append(torch.from_numpy(x).bfloat16().cuda())
    k, v = kv
    cache = FlashLoopCache(1, heads, 2, n)
    abi.fl_encode_base(cache.dims, cache.buf, 0, 0, k, v)
    want = cache.raw("brec", 0)[: heads * n // 64 * REC].view(heads, n // 64, REC)
    pair = Pair(1, n // 64 + 1, n // 64 + 1, heads)
    rows = lambda t: torch.cat([t, t[:, :1]], 1).transpose(0, 1)  # noqa: E731
    start, cu = pair.c.extend(i32([0]), i32([n + 1]))
    pair.c.append(0, i32([0]), start, cu, rows(k), rows(v))
    got = pair.c.pools[0].rec[pair.c.index.table[0, : n // 64].long()].transpose(0, 1)
    for t in range(heads):
        for j in range(n // 64):
            assert torch.equal(got[t, j], want[t, j]), (t, j)


@pytest.mark.parametrize("kv,n,active", [(1, 77, 1), (3, 700, 130), (2, 64 * 9, 300)])
def test_rows_read_back_feed_the_prefill_attention(kv, n, active):
    """A cached prefix read into [head][token] rows, and the attention of its last tokens over them."""
    g = gen(7, kv, n)
    pair = Pair(2, 16, 16, kv)
    pair.step([1], [n], g)
    k, v = torch.full((2, kv, n, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    place, pos = pair.c.places(i32([1]), i32([0]), i32([0, n]), n)
    paged.fl_paged_read(pair.c.index, pair.c.pools[0], place, k.transpose(0, 1), v.transpose(0, 1))
    for h in range(kv):
        for got, ref in zip((k, v), pair.o.keys_values(1, h)):
            assert torch.equal(got[h].cpu(), torch.from_numpy(ref.astype(np.float32)).bfloat16())
    q = bf16(g, kv, active, D)
    o = torch.full((kv, active, D), float("nan"), device="cuda")
    abi.fl_prefill_attn_sparse(q.cuda(), pos[n - active:].contiguous(), k, v, o)
    ref = fo.prefill_attention(f32(q), np.arange(n - active, n), f32(k), f32(v))
    # the prefill attention's own tolerance, per row (test_gpu_prefill.py)
    assert (np.abs(o.cpu().numpy() - ref).max(-1) <= 2e-3 * np.abs(ref).max(-1)).all()


# ------------------------------------------------------------------------------- attention
MIXED = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000, 1345, 20000, 9000, 3000]


@pytest.mark.parametrize("kv,group,max_pages,keep", [(2, 5, 460, 420), (1, 6, 900, 840), (4, 8, 320, 210), (2, 9, 460, 420),
                                                     (1, 12, 900, 840), (1, 17, 900, 840)])
def test_large_calls_of_many_heads_a_group(kv, group, max_pages, keep):
    """Groups above 4 where the call can hold more than 8 units a warp: eight heads a segment, in one
    segment and in several, every length, pieces cut between warps and between CTAs; the whole
    cache, the best blocks, and any blocks."""
    few = 8 * 12 * torch.cuda.get_device_properties(0).multi_processor_count
    assert len(MIXED) * kv * (keep + 4) > few and keep < max_pages
    g = gen(8, kv, group)
    pair, slots = random_cache(MIXED, max_pages, kv, group, 8 * kv + group)
    q = bf16(g, len(slots), kv * group, D, scale=1.5)
    o, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:2], float("nan"), device="cuda")
    pair.c.attend(0, i32(slots), q.cuda(), o, lse)
    check_attention(pair, slots, q, o, lse)
    again = torch.empty_like(o)
    pair.c.attend(0, i32(slots), q.cuda(), again)
    assert torch.equal(again, o)
    sel = pair.c.select(0, i32(slots), q.cuda(), keep)
    best = check_selection(pair, slots, q, sel, keep)
    r = np.random.default_rng(group)
    some = [[sorted(r.permutation(full(n))[: full(n) * 2 // 3].tolist()) for _ in range(kv)] for n in MIXED]
    rows = torch.tensor([[c + [-1] * (keep - len(c)) for c in head] for head in some], dtype=torch.int32, device="cuda")
    for chosen, picked in ((best, sel), (some, rows)):
        o.fill_(float("nan")), lse.fill_(float("nan"))
        paged.fl_paged_attn_decode(pair.c.index, pair.c.pools[0], i32(slots), q.cuda(), o, pair.c.ws, lse=lse, sel=picked)
        check_attention(pair, slots, q, o, lse, chosen)
    assert pair.c.status()[2] == 0


@pytest.mark.parametrize("group", [7, 11])
def test_large_calls_of_many_entries_and_heads(group):
    """The same kernels behind the block-wide scan of more than 128 entries, padded ones among them."""
    r = np.random.default_rng(group)
    lengths = r.integers(0, 400, 300).tolist()
    assert 300 * (46 + 4) > 8 * 12 * torch.cuda.get_device_properties(0).multi_processor_count
    pair, slots = random_cache(lengths, 46, 1, group, group)
    named = np.array(slots)
    named[r.random(300) < 0.1] = -1
    q = bf16(gen(9, group), 300, group, D, scale=1.5)
    o, lse = torch.full(q.shape, 7.0, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    pair.c.attend(0, i32(named), q.cuda(), o, lse)
    live = np.flatnonzero(named >= 0)
    check_attention(pair, named[live], q[live], o[live], lse[live])
    assert (o[named < 0] == 7).all() and (lse[named < 0] == 7).all()


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


# ------------------------------------------------------------------------------- selection
LONG = [64 * 515 + 9, 64 * 300, 64 * 257 + 64, 64 * 256 + 1, 64 * 130 + 5, 64 * 65 + 2, 64 * 64 + 2, 64 * 9, 70, 64, 0]


@pytest.mark.parametrize("max_pages", [257, 258, 520])
@pytest.mark.parametrize("kv,group,keep", [(1, 1, 1), (2, 4, 52), (1, 11, 64), (1, 2, 255), (3, 1, 256)])
def test_selection_of_long_requests(max_pages, kv, group, keep):
    """Requests of up to 515 blocks and short ones beside them, in tables on both sides of the
    width that decides how blocks are ordered, several chunks of 64 blocks a head."""
    lengths = [min(n, 64 * max_pages) for n in LONG]
    pair, slots = random_cache(lengths, max_pages, kv, group, max_pages + keep)
    q = bf16(gen(10, kv, group, keep), len(slots), kv * group, D, scale=1.5)
    check_selection(pair, slots, q, pair.c.select(0, i32(slots), q.cuda(), keep), keep)
    assert pair.c.status()[2] == 0


@pytest.mark.parametrize("max_pages,blocks", [(260, 64), (260, 258), (520, 257), (520, 515), (4100, 4001)])
@pytest.mark.parametrize("kinds", [1, 2, 7])
def test_equal_scores_over_many_blocks_go_to_the_lower_ones(max_pages, blocks, kinds):
    """Few different scores, ties across warps, chunks and passes: all equal, and a handful of values;
    from one block kept to all but one."""
    n = 64 * blocks + 3
    pair, slots = random_cache([n, n // 2, n], max_pages, 1, 2, blocks + kinds, kinds)
    q = bf16(gen(11, blocks, kinds), 3, 2, D)
    for keep in sorted({1, 5, 31, 64, blocks // 2, min(256, blocks - 1), blocks - 1}):
        check_selection(pair, slots, q, pair.c.select(0, i32(slots), q.cuda(), keep), keep)
    q[:] = 0                                    # every score is 0
    check_selection(pair, slots, q, pair.c.select(0, i32(slots), q.cuda(), 40), 40)


@pytest.mark.parametrize("max_pages", [250, 400])
def test_blocks_that_are_not_finite_are_the_last_taken(max_pages):
    pair, slots = random_cache([64 * 240 + 1, 64 * 100], max_pages, 2, 3, max_pages)
    r = np.random.default_rng(max_pages)
    ksz = pair.o.rec[..., 8704:].view(np.float16)
    for bad in (np.inf, -np.inf, np.nan):
        pages = r.permutation(len(ksz))[:60]
        ksz[pages, r.integers(0, 2, 60), r.integers(0, 256, 60)] = bad
    pair.c.pools[0].rec.copy_(torch.from_numpy(pair.o.rec))
    q = bf16(gen(12, max_pages), 2, 6, D)
    for keep in (3, 60, 230, 239):              # the last ones have to take some of them
        check_selection(pair, slots, q, pair.c.select(0, i32(slots), q.cuda(), keep), keep)


def test_selection_of_forty_requests():
    r = np.random.default_rng(40)
    lengths = r.integers(0, 64 * 90, 40).tolist()
    for max_pages in (95, 300):
        pair, slots = random_cache(lengths, max_pages, 2, 4, max_pages)
        named = np.array(slots)
        named[[4, 17, 39]] = -1
        q = bf16(gen(13), 40, 8, D, scale=1.5)
        sel = torch.full((40, 2, 12), -9, dtype=torch.int32, device="cuda")
        paged.fl_paged_select(pair.c.index, pair.c.pools[0], i32(named), q.cuda(), sel, pair.c.ws)
        live = np.flatnonzero(named >= 0)
        check_selection(pair, named[live], q[live], sel[torch.from_numpy(live).cuda()], 12)
        assert (sel[[4, 17, 39]] == -9).all()


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
