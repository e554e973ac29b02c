"""The paged cache on the GPU against its oracle: tables and slot maps, appended records byte
for byte, rows read back, attention over whole caches and over selected blocks, and all of
them together as a serving loop uses them."""
import numpy as np
import pytest
import torch

from oracle.paged_oracle import D, PAGE, full
from pagedhelpers import Pair, bf16, check_attention, f32, i32
from quantized_kv_attention_int4_b200 import abi, paged

pytestmark = pytest.mark.gpu


def gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 7919 * int(k) for i, k in enumerate(key)) + 17)


# ------------------------------------------------------------------------------- tables
@pytest.mark.parametrize("slots,max_pages,pages,batch", [(4, 5, 12, 4), (700, 3, 900, 300), (3000, 2, 2500, 2600)])
def test_tables_follow_the_oracle_through_random_steps(slots, max_pages, pages, batch):
    r = np.random.default_rng(slots)
    pair = Pair(slots, max_pages, pages, 1)
    x, o = pair.c.index, pair.o
    for step in range(6):
        sl = r.permutation(slots)[:batch]
        sl[r.random(batch) < 0.1] = -1
        n = r.integers(0, 90, batch)
        if step == 3:
            n[r.random(batch) < 0.05] = -3
            n[r.random(batch) < 0.05] = 64 * max_pages + 1
            sl[r.random(batch) < 0.02] = slots + 5
            sl[batch // 2] = sl[0]
            sl[-1] = sl[1]
        if step == 4 and batch == slots:
            sl = None
        start, cu = pair.c.extend(None if sl is None else i32(sl), i32(n))
        ostart, ocu = o.extend(sl, n)
        assert start.tolist() == ostart.tolist() and cu.tolist() == ocu.tolist()
        pair.same_index()
        t = int(ocu[-1])
        place = torch.full((t + 5,), -7, dtype=torch.int32, device="cuda")
        pos = place.clone()
        paged.fl_paged_slot_map(x, None if sl is None else i32(sl), start, cu, place, pos)
        oplace, opos = o.slot_map(sl, ostart, ocu, t + 5)
        assert place.tolist() == oplace.tolist() and pos.tolist() == opos.tolist()
        back = r.permutation(slots)[: batch // 3 + 1]
        back[back % 7 == 0] = -1
        if step == 2:
            back[-1] = back[0]
        pair.c.release(i32(back))
        o.release(back, len(back))
        pair.same_index()
    code, detail, count = pair.c.status()
    assert count == len(o.errors) and (code, detail) in o.errors
    assert pair.c.status()[2] == 0


@pytest.mark.parametrize("pages", [9000, 2500])
def test_few_requests_of_many_pages(pages):
    r = np.random.default_rng(12)
    slots, max_pages = 110, 210
    pair = Pair(slots, max_pages, pages, 1)
    for step in range(5):
        sl = r.permutation(slots)[:100]
        sl[3], sl[60] = -1, sl[10]
        n = r.integers(0, 64 * max_pages // 2, 100)
        n[r.random(100) < 0.3] = 1
        start, cu = pair.c.extend(i32(sl), i32(n))
        ostart, ocu = pair.o.extend(sl, n)
        assert start.tolist() == ostart.tolist() and cu.tolist() == ocu.tolist()
        pair.same_index()
        back = r.permutation(slots)[:50 + step]
        back[7], back[20] = -1, back[9]
        pair.c.release(i32(back))
        pair.o.release(back, len(back))
        pair.same_index()
    code, detail, count = pair.c.status()
    assert count == len(pair.o.errors) and (code, detail) in pair.o.errors
    assert {c for c, _ in pair.o.errors} >= {paged.FL_DEV_SLOT_TWICE, paged.FL_DEV_TOO_LONG if pages == 9000 else paged.FL_DEV_NO_PAGE}


def test_one_long_request_and_an_empty_batch():
    pair = Pair(2, 16384, 16390, 1, max_batch=1)
    n = 16384 * 64
    start, cu = pair.c.extend(i32([1]), i32([n]))
    assert start.tolist() == [0] and cu.tolist() == [0, n]
    assert pair.c.index.table[1].tolist() == list(range(16384)) and pair.c.index.n_free.item() == 6
    assert pair.c.extend(i32([1]), i32([1]))[0].tolist() == [-1] and pair.c.status()[0] == paged.FL_DEV_TOO_LONG
    start, cu = pair.c.extend(i32([]), i32([]))
    assert cu.tolist() == [0]
    place, pos = pair.c.places(i32([1]), i32([n - 70]), i32([0, 71]), 72)
    assert place.tolist() == [(16382 + (i + 58) // 64) * 64 + (i + 58) % 64 for i in range(6)] + [
        (16390 + 1) * 64 + i for i in range(64)] + [-1, -1]
    assert pos.tolist() == list(range(n - 70, n + 1)) + [-1]
    pair.c.release(i32([1]))
    assert pair.c.index.n_free.item() == 16390 and pair.c.index.free_pages[-1].item() == 16383


# ------------------------------------------------------------------------------- append and read
@pytest.mark.parametrize("kv", [1, 3])
def test_append_writes_the_oracles_bytes_whatever_the_pieces(kv):
    g = gen(3, kv)
    pair = Pair(6, 8, 40, kv)
    steps = [([0, 1, 2, 3, 4], [1, 63, 64, 65, 200]), ([4, 2, 1, 0], [1, 1, 1, 0]), ([3, 0, -1, 1], [64, 127, 9, 128]),
             (None, [1, 2, 3, 4, 5, 6]), ([5, 4], [58, 64]), ([5], [1])]
    for slots, n in steps:
        pair.step(slots, n, g)
        pair.same_index()
        pair.same_bytes()
    assert pair.c.status()[2] == 0
    # every token back, as BF16
    n = pair.o.length
    cu = np.concatenate([[0], np.cumsum(n)])
    place, _ = pair.c.places(None, i32(np.zeros(6)), i32(cu), int(cu[-1]) + 3)
    k, v = pair.c.read(0, place)
    for s in range(6):
        for h in range(kv):
            ok, ov = pair.o.keys_values(s, h)
            for got, ref in ((k, ok), (v, ov)):
                ref = torch.from_numpy(ref.astype(np.float32)).to(torch.bfloat16)
                assert torch.equal(got[cu[s]: cu[s + 1], h].cpu(), ref)
    assert not k[cu[-1]:].any() and not v[cu[-1]:].any()


def test_append_leaves_other_rows_alone_and_takes_strides():
    g = gen(4)
    pair = Pair(3, 4, 8, 2)
    pool = pair.c.pools[0]
    x = bf16(g, 100, 3, 4, 136)                 # k and v are slices of one projection's output
    k, v = x[:, 0, 1:3, :128], x[:, 1, 1:3, :128]
    dev = x.cuda()
    start, cu = pair.c.extend(i32([2, 0]), i32([70, 20]))
    pair.o.extend([2, 0], [70, 20])
    pair.c.append(0, i32([2, 0]), start, cu, dev[:, 0, 1:3, :128], dev[:, 1, 1:3, :128])
    pair.o.append([2, 0], [0, 0], [0, 70, 90], f32(k), f32(v))
    pair.same_bytes()
    assert torch.isnan(pool.tail_k[1]).all() and torch.isnan(pool.tail_k[2, :, 6:]).all()
    assert torch.isnan(pool.tail_v[0, :, 20:]).all()
    assert not pool.rec[1:].any()               # page 0 is the only one that filled up
    # reading into strided rows: those of place -1 stay
    out = torch.full((5, 2, 3, 160), 9.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = out[:, 0, :2, :128], out[:, 1, :2, :128]
    paged.fl_paged_read(pair.c.index, pool, i32([63, -1, 0, (8 + 2) * 64 + 5, -1]), ko, vo)
    ok, ov = pair.o.keys_values(2, 1)
    for i, t in ((0, 63), (2, 0), (3, 69)):
        assert torch.equal(ko[i, 1].cpu().float(), torch.from_numpy(ok[t].astype(np.float32)).bfloat16().float())
        assert torch.equal(vo[i, 1].cpu().float(), torch.from_numpy(ov[t].astype(np.float32)).bfloat16().float())
    assert (out[[1, 4]] == 9).all() and (out[:, :, 2] == 9).all() and (out[..., 128:] == 9).all()


def test_groups_of_equal_tiny_and_large_values_are_exact():
    pair = Pair(1, 4, 4, 1)
    n = 64 * 3 + 1
    g = gen(5)
    k, v = bf16(g, n, 1, D), bf16(g, n, 1, D)
    k[:64, 0, :32] = 0.75                       # scale 0
    k[:64, 0, 32:64] *= 2.0 ** -20              # scales below the smallest 16-bit number
    k[:64, 0, 64:96] *= 2.0 ** -13              # subnormal scales
    k[64:128] *= 8192.0
    v[:8, 0, :64] = -3.0
    v[8:16] *= 2.0 ** -14
    v[64:128] *= 8192.0
    v[128:192, 0, 7] = 0.5 * torch.arange(64).bfloat16()
    k[128:192, 0, 7] = 0.5 * torch.arange(64).bfloat16()   # quotients near halves
    start, cu = pair.c.extend(i32([0]), i32([n]))
    pair.c.append(0, i32([0]), start, cu, k.cuda(), v.cuda())
    s, c = pair.o.extend([0], [n])
    pair.o.append([0], s, c, f32(k), f32(v))
    pair.same_bytes()


def test_codes_at_every_half_are_the_rounded_divisions():
    """Integers over every spread 1 .. 130: quotients (x - z) / s at and next to halves."""
    m = 130
    pair = Pair(1, m + 1, m + 1, 1)
    k = torch.zeros(64 * m + 1, 1, D, dtype=torch.bfloat16)
    for i in range(m):
        k[64 * i: 64 * i + 64, 0] = (torch.arange(64)[:, None] * torch.arange(1, D + 1) % (i + 2)).bfloat16() * (1 + i / 64)
    start, cu = pair.c.extend(i32([0]), i32([len(k)]))
    pair.c.append(0, i32([0]), start, cu, k.cuda(), k.cuda())
    s, c = pair.o.extend([0], [len(k)])
    pair.o.append([0], s, c, f32(k), f32(k))
    pair.same_bytes()


def near_half_groups(r, n):
    """BF16 values [n][64] whose quotients (x - z) / s lie at, and a few units in the last place
    beside, halves: among them groups with z = -(a + 0.5) s, where tiny values do."""
    s = np.exp2(r.integers(-18, 9, (n, 1))) * (1 + r.integers(0, 8, (n, 1)) / 8)
    z = -(r.integers(0, 15, (n, 1)) + r.choice([0.0, 0.5], (n, 1))) * s * r.choice([1, 1, 1, 0, 40], (n, 1))
    x = torch.from_numpy(z + (r.integers(0, 15, (n, 64)) + 0.5) * s).bfloat16()
    x = (x.view(torch.int16) + torch.from_numpy(r.integers(-2, 3, (n, 64))).short()).view(torch.bfloat16)
    tiny = torch.from_numpy(r.choice([0.0, -0.0, 1e-40, -1e-40, 1e-30, -1e-30, 1e-8, -1e-8], (n, 64))).bfloat16()
    x = torch.where(torch.from_numpy(r.random((n, 64)) < 0.3), tiny, x)
    x[:, 0], x[:, 63] = torch.from_numpy(z[:, 0]).bfloat16(), torch.from_numpy(z[:, 0] + 15 * s[:, 0]).bfloat16()
    x = torch.where(x.isfinite(), x, 0.0)
    x[::97] -= 66560.0                           # zero beyond the 16-bit numbers, a finite scale
    return x


def test_codes_beside_halves_are_the_rounded_divisions():
    r = np.random.default_rng(31)
    m = 120
    pair = Pair(1, m + 1, m + 1, 1)
    k = near_half_groups(r, m * D).reshape(m, D, 64).transpose(1, 2).reshape(m * 64, 1, D)
    v = near_half_groups(r, m * 64 * 2).reshape(m * 64, 1, D)
    k, v = (torch.cat([t, torch.zeros(1, 1, D, dtype=torch.bfloat16)]).contiguous() for t in (k, v))
    start, cu = pair.c.extend(i32([0]), i32([len(k)]))
    pair.c.append(0, i32([0]), start, cu, k.cuda(), v.cuda())
    s, c = pair.o.extend([0], [len(k)])
    pair.o.append([0], s, c, f32(k), f32(v))

    def plain(rec):
        # the least of a group that holds both zeros is either of them: -0 as 0 in the scale words
        sz = rec[..., 8192:].view(np.uint16)
        sz[sz == 0x8000] = 0
        return rec

    got, want = plain(pair.c.pools[0].rec.cpu().numpy()), plain(pair.o.rec.copy())
    for j in range(m):
        assert np.array_equal(got[pair.o.table[0, j]], want[pair.o.table[0, j]]), j


def test_append_skips_rows_beyond_its_input_and_bad_pages():
    g = gen(6)
    pair = Pair(3, 4, 9, 1)
    start, cu = pair.c.extend(i32([0, 1]), i32([70, 70]))
    k = bf16(g, 100, 1, D).cuda()               # the second request's rows pass the end
    pair.c.append(0, i32([0, 1]), start, cu, k, k)
    assert pair.c.status()[:2] == [paged.FL_DEV_COUNT, 1]
    assert torch.isnan(pair.c.pools[0].tail_k[1]).all()
    pair.c.index.table[1, 0] = 9                # a page outside the pool
    pair.c.append(0, i32([1]), i32([0]), i32([0, 70]), k, k)
    assert pair.c.status()[:2] == [paged.FL_DEV_PAGE_RANGE, 0]
    assert torch.equal(pair.c.pools[0].tail_k[1, 0, :6], k[64:70, 0])
    pair.c.append(0, i32([7]), i32([0]), i32([0, 70]), k, k)
    assert pair.c.status()[:2] == [paged.FL_DEV_SLOT_RANGE, 0]
    out = torch.zeros(2, 1, D, dtype=torch.bfloat16, device="cuda")
    paged.fl_paged_read(pair.c.index, pair.c.pools[0], i32([(9 + 3) * 64, -5]), out, out.clone())
    assert pair.c.status()[0] == paged.FL_DEV_PAGE_RANGE and not out.any()


def test_a_bad_page_is_told_once_a_block_and_head():
    pair = Pair(2, 3, 6, 3)
    start, cu = pair.c.extend(i32([1, 0]), i32([10, 129]))
    pair.c.index.table[0, 1] = 6
    k = bf16(gen(8), 139, 3, D).cuda()
    pair.c.append(0, i32([1, 0]), start, cu, k, k)
    assert pair.c.status() == [paged.FL_DEV_PAGE_RANGE, 1, 3]
    assert torch.equal(pair.c.pools[0].tail_v[0, :, 0], k[138])


# ------------------------------------------------------------------------------- attention
LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000, 1345]


def filled(lengths, kv, group, g, scale=1.0, spare=2):
    pair = Pair(len(lengths) + spare, max(-(-max(lengths) // PAGE), 1) + 1, sum(-(-n // PAGE) for n in lengths) + 3, kv, kv * group)
    slots = torch.randperm(len(lengths) + spare, generator=g)[: len(lengths)].tolist()
    pair.step(slots, lengths, g, scale)
    return pair, slots


@pytest.mark.parametrize("kv,group", [(1, 1), (2, 2), (3, 3), (2, 4), (1, 5), (2, 7), (1, 8), (1, 9), (1, 12), (1, 17)])
def test_attention_matches_the_oracle_at_every_length(kv, group):
    g = gen(7, kv, group)
    pair, slots = filled(LENGTHS, kv, group, g)
    q = bf16(g, len(slots), kv * group, D, scale=1.5)
    o = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    pair.c.attend(0, i32(slots), q.cuda(), o, lse)
    check_attention(pair, slots, q, o, lse)
    assert not o[0].any()                       # the request of no tokens
    again = torch.empty_like(o)
    pair.c.attend(0, i32(slots), q.cuda(), again)
    assert torch.equal(again, o)
    assert pair.c.status()[2] == 0


@pytest.mark.parametrize("lengths,kv,group", [([20000], 1, 1), ([20000, 3, 9000], 2, 4), ([4096] * 3 + [1] * 40, 4, 8)])
def test_long_and_ragged_batches(lengths, kv, group):
    g = gen(8, len(lengths), kv)
    pair, slots = filled(lengths, kv, group, g)
    q = bf16(g, len(slots), kv * group, D, scale=1.5)
    o = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    pair.c.attend(0, i32(slots), q.cuda(), o, lse)
    check_attention(pair, slots, q, o, lse)


@pytest.mark.parametrize("scale", [2.0 ** -9, 2.0 ** -4, 30.0, 1000.0])
def test_small_and_large_keys_and_values(scale):
    """Scales far from 1: a hot softmax (scores of hundreds) and a flat one."""
    g = gen(9, int(scale * 512))
    pair, slots = filled([700, 70, 64, 5], 2, 4, g, scale)
    q = bf16(g, 4, 8, D, scale=1.0 if scale < 100 else 2.0 ** -9)
    o = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    pair.c.attend(0, i32(slots), q.cuda(), o, lse)
    check_attention(pair, slots, q, o, lse)


def test_queries_of_any_size_in_one_call():
    """Zero, tiny and huge queries beside ordinary ones in one group."""
    g = gen(10)
    pair, slots = filled([400, 90], 1, 6, g)
    q = bf16(g, 2, 6, D)
    q[:, 0] = 0
    q[:, 1] *= 2.0 ** -60
    q[:, 2] *= 2.0 ** -10
    q[:, 3] *= 100.0
    q[:, 4, 1:] = 0                             # one channel alone
    q[:, 5, ::2] *= 2.0 ** -16
    o = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    pair.c.attend(0, i32(slots), q.cuda(), o, lse)
    check_attention(pair, slots, q, o, lse)


def test_blocks_of_very_different_scales_in_one_request():
    """Keys and values that grow and shrink by 2^12 from block to block."""
    g = gen(11)
    pair = Pair(1, 12, 12, 1, 4)
    for i, e in enumerate((0, -12, 6, -6, 0, 8, -10, 0, 3)):
        n = 64
        k = (bf16(g, n, 1, D).float() * 2.0 ** (e // 2)).bfloat16()
        v = (bf16(g, n, 1, D).float() * 2.0 ** e).bfloat16()
        start, cu = pair.c.extend(i32([0]), i32([n]))
        pair.c.append(0, i32([0]), start, cu, k.cuda(), v.cuda())
        s, c = pair.o.extend([0], [n])
        pair.o.append([0], s, c, f32(k), f32(v))
    q = bf16(g, 1, 4, D, scale=0.25)
    q[0, 3] *= 2.0 ** -6                        # flat: every block counts
    o = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    pair.c.attend(0, i32([0]), q.cuda(), o, lse)
    check_attention(pair, [0], q, o, lse)


def test_padded_entries_strides_and_shared_requests():
    g = gen(12)
    pair, slots = filled([130, 70, 64, 1], 2, 3, g)
    named = [slots[1], -1, slots[0], slots[0], -1, slots[3]]       # one request may stand twice
    wide = bf16(g, 6, 8, 144)
    q = wide[:, 1:7, :128]
    dev = wide.cuda()
    o = torch.full((6, 7, 160), 5.0, device="cuda")
    lse = torch.full((6, 6), 5.0, device="cuda")
    pair.c.attend(0, i32(named), dev[:, 1:7, :128], o[:, :6, :128], lse)
    live = [0, 2, 3, 5]
    check_attention(pair, [named[i] for i in live], q[live], o[live][:, :6, :128], lse[live])
    assert (o[[1, 4]] == 5).all() and (lse[[1, 4]] == 5).all()
    assert (o[:, 6] == 5).all() and (o[..., 128:] == 5).all()
    assert pair.c.status()[2] == 0
    pair.c.attend(0, i32([99, slots[0]]), dev[:2, 1:7, :128])
    assert pair.c.status()[:2] == [paged.FL_DEV_SLOT_RANGE, 0]


def test_infinite_and_nan_rows_stay_where_they_belong():
    """A NaN or infinite key of one request spoils that request alone; rows behind a tail's end
    hold NaN in every test here and spoil nothing."""
    g = gen(13)
    pair, slots = filled([70, 75, 80], 1, 2, g)
    pool = pair.c.pools[0]
    q = bf16(g, 3, 2, D)
    clean, lse = torch.empty(q.shape, device="cuda"), torch.empty(3, 2, device="cuda")
    pair.c.attend(0, i32(slots), q.cuda(), clean, lse)
    check_attention(pair, slots, q, clean, lse)
    pool.tail_k[slots[1], 0, 3, 5] = float("nan")
    pool.tail_v[slots[2], 0, 2, 7] = float("inf")
    o = torch.empty_like(clean)
    pair.c.attend(0, i32(slots), q.cuda(), o)
    assert torch.equal(o[0], clean[0]) and torch.isnan(o[1]).all()
    assert torch.isinf(o[2, :, 7]).all() and torch.allclose(o[2, :, 8:], clean[2, :, 8:], rtol=1e-5, atol=1e-6)


# ------------------------------------------------------------------------------- selection
@pytest.mark.parametrize("kv,group,keep", [(1, 1, 1), (2, 4, 5), (3, 1, 16), (1, 8, 3), (1, 11, 7), (2, 2, 500)])
def test_selection_and_attention_over_it(kv, group, keep):
    g = gen(14, kv, group, keep)
    lengths = LENGTHS + [64 * 40 + 7]
    pair, slots = filled(lengths, kv, group, g)
    q = bf16(g, len(slots), kv * group, D, scale=1.5)
    qn = q.double().numpy()
    sel = pair.c.select(0, i32(slots), q.cuda(), keep).cpu().numpy()
    chosen = []
    for b, s in enumerate(slots):
        chosen.append([])
        for h in range(kv):
            want = pair.o.select(s, h, qn[b, h * group: (h + 1) * group], keep)
            assert sel[b, h].tolist() == want + [-1] * (keep - len(want)), (b, h)
            chosen[-1].append(want)
    o = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    paged.fl_paged_attn_decode(pair.c.index, pair.c.pools[0], i32(slots), q.cuda(), o, pair.c.ws, lse=lse,
                               sel=torch.from_numpy(sel).cuda())
    check_attention(pair, slots, q, o, lse, chosen)
    assert torch.equal(pair.c.attend(0, i32(slots), q.cuda(), keep=keep), o)
    assert pair.c.status()[2] == 0


def test_equal_scores_go_to_the_lower_block_and_padded_rows_stay():
    g = gen(15)
    pair = Pair(2, 40, 80, 1)
    k = bf16(g, 64, 1, D).repeat(33, 1, 1)      # every block is the same
    k[64 * 20: 64 * 21] += 1.0
    n = 64 * 32 + 3
    start, cu = pair.c.extend(i32([1]), i32([n]))
    pair.c.append(0, i32([1]), start, cu, k[:n].cuda(), k[:n].cuda())
    q = torch.ones(2, 1, D, dtype=torch.bfloat16, device="cuda")
    sel = torch.full((2, 1, 6), -9, dtype=torch.int32, device="cuda")
    paged.fl_paged_select(pair.c.index, pair.c.pools[0], i32([-1, 1]), q, sel, pair.c.ws)
    assert sel.tolist() == [[[-9] * 6], [[0, 1, 2, 3, 4, 20]]]
    q[:] = 0                                    # every score is 0
    paged.fl_paged_select(pair.c.index, pair.c.pools[0], i32([-1, 1]), q, sel, pair.c.ws)
    assert sel[1, 0].tolist() == [0, 1, 2, 3, 4, 5]


def test_selected_blocks_that_are_none_are_skipped_and_told():
    g = gen(16)
    pair, slots = filled([64 * 5 + 9], 1, 1, g)
    q = bf16(g, 1, 1, D)
    o, lse = torch.empty(1, 1, D, device="cuda"), torch.empty(1, 1, device="cuda")
    for sel, live, err in (([0, 3, -1, -1], [0, 3], 0), ([-1, -1], [], 0), ([2, 5], [2], paged.FL_DEV_SEL_BLOCK),
                           ([-4, 1], [1], paged.FL_DEV_SEL_BLOCK), ([10 ** 9, 0, 4], [0, 4], paged.FL_DEV_SEL_BLOCK)):
        paged.fl_paged_attn_decode(pair.c.index, pair.c.pools[0], i32(slots), q.cuda(), o, pair.c.ws, lse=lse,
                                   sel=i32([[sel]]))
        check_attention(pair, slots, q, o, lse, [[live]])
        assert pair.c.status()[0] == err


def test_bad_tables_and_lengths_are_told_and_read_nothing():
    g = gen(17)
    pair, slots = filled([64 * 6 + 9, 30], 1, 2, g)
    x = pair.c.index
    q = bf16(g, 2, 2, D).cuda()
    s = slots[0]
    x.table[s, 2] = x.pages
    o, lse = torch.empty(2, 2, D, device="cuda"), torch.empty(2, 2, device="cuda")
    pair.c.attend(0, i32(slots), q, o, lse)
    assert pair.c.status()[:2] == [paged.FL_DEV_PAGE_RANGE, 0]
    check_attention(pair, slots, q.cpu(), o, lse, [[[0, 1, 3, 4, 5]], [[]]])
    pair.c.select(0, i32(slots), q, 2)
    assert pair.c.status()[0] == paged.FL_DEV_PAGE_RANGE
    for bad in (-5, 64 * x.max_pages + 1, 2 ** 31 - 1):
        x.length[s] = bad
        pair.c.attend(0, i32(slots), q, o, lse)
        assert pair.c.status()[0] == paged.FL_DEV_TOO_LONG
        assert not o[0].any() and torch.isneginf(lse[0]).all()
        assert pair.c.select(0, i32(slots), q, 2)[0].tolist() == [[-1, -1]]
        pair.c.status()


# ------------------------------------------------------------------------------- together
def test_a_serving_loop_with_requests_that_come_and_go():
    """Admit, decode, attend dense and sparse, finish, re-admit on the same pages, two planes."""
    g = gen(18)
    r = np.random.default_rng(18)
    kv, group, slots = 2, 4, 5
    pair = Pair(slots, 8, 22, kv, kv * group)
    other = paged.PagedPool.empty(pair.c.index, kv)     # a second plane on the same index
    live = {}
    for step in range(40):
        for s in [s for s, left in live.items() if left == 0]:
            pair.c.release(i32([s]))
            pair.o.release([s], 1)
            del live[s]
        batch, n_new = list(live), [1] * len(live)
        for s in range(slots):
            if s not in live and r.random() < 0.4:
                n = int(r.integers(1, 200))
                if sum(-(-int(pair.o.length[t]) // PAGE) + 1 for t in range(slots)) + -(-n // PAGE) <= 20:
                    batch.append(s)
                    n_new.append(n)
                    live[s] = int(r.integers(3, 90))
        order = r.permutation(len(batch))
        batch, n_new = [batch[i] for i in order] + [-1], [n_new[i] for i in order] + [0]
        start, cu = pair.step(batch, n_new, g)
        t = max(int(cu[-1].item()), 1)
        k2 = bf16(g, t, kv, D).cuda()
        paged.fl_paged_append(pair.c.index, other, i32(batch), start, cu, k2, k2)
        for s in live:
            live[s] -= 1
        if step % 4 == 3:
            q = bf16(g, len(batch), kv * group, D, scale=1.5)
            o = torch.empty(q.shape, device="cuda")
            lse = torch.empty(q.shape[:2], device="cuda")
            pair.c.attend(0, i32(batch), q.cuda(), o, lse)
            m = len(batch) - 1
            check_attention(pair, batch[:m], q[:m], o[:m], lse[:m])
            pair.c.attend(0, i32(batch), q.cuda(), o, lse, keep=2)
            qn = q.double().numpy()
            chosen = [[pair.o.select(s, h, qn[b, h * group: (h + 1) * group], 2) for h in range(kv)]
                      for b, s in enumerate(batch[:m])]
            check_attention(pair, batch[:m], q[:m], o[:m], lse[:m], chosen)
    pair.same_index()
    pair.same_bytes()
    assert pair.c.status()[2] == 0 and not pair.o.errors


def test_a_captured_step_replays_on_grown_requests():
    """One decode step (extend, slot map, append, select, attention) captured into a CUDA graph
    and replayed: lengths, tables and selections move on inside the graph."""
    g = gen(19)
    kv, group, n = 2, 2, 3
    pair = Pair(n, 6, 18, kv, kv * group)
    pair.step(None, [60, 126, 64 * 4 - 2], g)
    steps = 8
    ks, vs, qs = bf16(g, steps, n, kv, D), bf16(g, steps, n, kv, D), bf16(g, steps, n, kv * group, D)
    k, v, q = torch.empty_like(ks[0], device="cuda"), torch.empty_like(vs[0], device="cuda"), torch.empty_like(qs[0], device="cuda")
    ones, slots = i32([1] * n), i32(range(n))
    start, cu, pos = i32([0] * n), i32([0] * (n + 1)), i32([0] * n)
    o, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    so, slse = torch.empty_like(o), torch.empty_like(lse)
    sel = torch.full((n, kv, 1), -1, dtype=torch.int32, device="cuda")
    c = pair.c

    def step():
        paged.fl_paged_extend(c.index, slots, ones, start, cu)
        paged.fl_paged_slot_map(c.index, slots, start, cu, None, pos)
        paged.fl_paged_append(c.index, c.pools[0], slots, start, cu, k, v)
        paged.fl_paged_attn_decode(c.index, c.pools[0], slots, q, o, c.ws, lse=lse)
        paged.fl_paged_select(c.index, c.pools[0], slots, q, sel, c.ws)
        paged.fl_paged_attn_decode(c.index, c.pools[0], slots, q, so, c.ws, lse=slse, sel=sel)

    def check(i):
        s, ocu = pair.o.extend(None, [1] * n)
        pair.o.append(None, s, ocu, f32(ks[i]), f32(vs[i]))
        assert pos.tolist() == s.tolist()
        check_attention(pair, None, qs[i], o, lse)
        qn = qs[i].double().numpy()
        chosen = [[pair.o.select(b, h, qn[b, h * group: (h + 1) * group], 1) for h in range(kv)] for b in range(n)]
        check_attention(pair, None, qs[i], so, slse, chosen)

    k.copy_(ks[0]), v.copy_(vs[0]), q.copy_(qs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, steps):
        k.copy_(ks[i]), v.copy_(vs[i]), q.copy_(qs[i])
        graph.replay()
        torch.cuda.synchronize()
        check(i)
    pair.same_bytes()
    assert c.status()[2] == 0


def test_captured_calls_behind_copies_and_joined_streams():
    """Captured behind a memory set, with two streams forked and joined (each with a workspace and a
    plane of its own), and replayed: the calls' programmatic launches keep every dependency."""
    g = gen(21)
    pair, slots = filled([700, 64, 130], 2, 4, g)
    c = pair.c
    other = paged.PagedPool.empty(c.index, 2)
    other.rec.copy_(c.pools[0].rec)
    other.tail_k.copy_(c.pools[0].tail_k), other.tail_v.copy_(c.pools[0].tail_v)
    ws2 = paged.workspace(c.index, other, 3, 8)
    sl = i32(slots)
    q = bf16(g, 3, 8, D, scale=1.5).cuda()
    ref, sref = c.attend(0, sl, q), c.attend(0, sl, q, keep=3)
    o1, o2, o3 = (torch.empty_like(ref) for _ in range(3))
    sel = torch.full((3, 2, 3), -1, dtype=torch.int32, device="cuda")
    place = torch.empty(64, dtype=torch.int32, device="cuda")
    k, v = torch.empty(64, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(64, 2, D, dtype=torch.bfloat16, device="cuda")
    begin, cu = i32([3, 0, 0]), i32([0, 64, 64, 64])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        paged.fl_paged_workspace_init(c.ws)
        o1.zero_()
        paged.fl_paged_attn_decode(c.index, c.pools[0], sl, q, o1, c.ws)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            paged.fl_paged_attn_decode(c.index, other, sl, q, o2, ws2)
            paged.fl_paged_slot_map(c.index, sl, begin, cu, place, None)
        paged.fl_paged_select(c.index, c.pools[0], sl, q, sel, c.ws)
        main.wait_stream(side)
        paged.fl_paged_read(c.index, other, place, k, v)
        paged.fl_paged_attn_decode(c.index, c.pools[0], sl, q, o3, c.ws, sel=sel)
    rows = torch.from_numpy(pair.o.keys_values(slots[0], 1)[0][3:67].astype(np.float32)).bfloat16()
    for _ in range(3):
        for t in (o1, o2, o3, k, v):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, ref) and torch.equal(o2, ref) and torch.equal(o3, sref)
        assert torch.equal(k[:, 1].cpu(), rows)


def test_many_entries_take_the_other_scan():
    """Beyond 128 entries a call scans its lengths block-wide: the same results, padded entries
    and requests of no tokens among them."""
    g = gen(22)
    r = np.random.default_rng(22)
    lengths = [int(n) for n in r.integers(0, 150, 300)]
    pair, slots = filled(lengths, 1, 2, g)
    q = bf16(g, 300, 2, D)
    o, lse = torch.empty(300, 2, D, device="cuda"), torch.empty(300, 2, device="cuda")
    named = np.array(slots)
    named[r.random(300) < 0.1] = -1
    o.fill_(7.0), lse.fill_(7.0)
    pair.c.attend(0, i32(named), q.cuda(), o, lse)
    live = [i for i in range(300) if named[i] >= 0]
    check_attention(pair, named[live], q[live], o[live], lse[live])
    assert (o[named < 0] == 7).all() and (lse[named < 0] == 7).all()
    first = torch.empty(100, 2, D, device="cuda")   # a part of it through the other path
    pair.c.attend(0, i32(slots[:100]), q[:100].cuda(), first)
    second = torch.empty(300, 2, D, device="cuda")
    pair.c.attend(0, i32(slots), q.cuda(), second)
    assert torch.allclose(first, second[:100], rtol=1e-5, atol=1e-6)


def test_calls_on_a_stream_of_their_own():
    g = gen(20)
    pair, slots = filled([500, 90], 2, 2, g)
    q = bf16(g, 2, 4, D).cuda()
    ref = pair.c.attend(0, i32(slots), q)
    sl = i32(slots)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = torch.empty(q.shape, device="cuda")
    paged.fl_paged_attn_decode(pair.c.index, pair.c.pools[0], sl, q, o, pair.c.ws, stream=side)
    side.synchronize()
    assert torch.equal(o, ref)


def test_binding_checks_shapes_strides_and_workspaces():
    pair = Pair(3, 2, 6, 2, 4)
    c = pair.c
    q, o = torch.zeros(3, 4, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 4, D, device="cuda")
    att = lambda **k: paged.fl_paged_attn_decode(c.index, c.pools[0], k.get("slots"), k.get("q", q), k.get("o", o),  # noqa: E731
                                                 k.get("ws", c.ws), lse=k.get("lse"), sel=k.get("sel"))
    with pytest.raises(TypeError):
        att(q=q.float())
    with pytest.raises(ValueError):
        att(q=q[..., :64])
    with pytest.raises(ValueError):
        att(o=o[:2])
    with pytest.raises(ValueError):
        att(slots=i32([0, 1]))
    with pytest.raises(ValueError):
        att(lse=torch.zeros(3, 3, device="cuda"))
    with pytest.raises(ValueError):
        att(sel=torch.zeros(3, 4, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(abi.FlashLoopError) as e:
        att(ws=c.ws[: paged.WS_HEAD])
    assert e.value.status == abi.FL_ERR_WORKSPACE
    with pytest.raises(abi.FlashLoopError) as e:
        att(q=torch.zeros(3, 3, D, dtype=torch.bfloat16, device="cuda"), o=o[:, :3])
    assert e.value.status == abi.FL_ERR_INVALID
    k = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
    s, cu = i32([0]), i32([0, 4])
    with pytest.raises(ValueError):
        paged.fl_paged_append(c.index, c.pools[0], i32([0]), s, cu, k, k[:3])
    with pytest.raises(ValueError):
        paged.fl_paged_append(c.index, c.pools[0], i32([0]), s, i32([0]), k, k)
    with pytest.raises(ValueError):
        paged.fl_paged_append(c.index, c.pools[0], i32([0]), s, cu, k[:, :1], k[:, :1])
    with pytest.raises(ValueError):
        paged.fl_paged_read(c.index, c.pools[0], i32([0]), k, k)
    small = paged.PagedPool(c.pools[0].rec[:4], c.pools[0].tail_k, c.pools[0].tail_v)
    with pytest.raises(ValueError, match="pages and slots"):
        paged.fl_paged_read(c.index, small, i32([0] * 4), k, k)
