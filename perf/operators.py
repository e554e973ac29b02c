"""The operators of the paged INT4 key-value cache, as plain torch operations and as the framework's calls.

The cache serves many requests at once.  A request sits in a row ("slot") of a block table;
block j of a request is 64 tokens whose keys and values lie in page table[slot][j] of a pool, one
9216-byte group record per (page, key-value head); the last 1..64 tokens of a request are BF16
rows of the slot's tail.  Five operators:

  index    pages taken and given back, lengths, and the place of every token (slot map)
  append   new keys and values into the cache: full blocks as INT4 records, the rest into the tail
  read     cached tokens back as BF16 rows, through a slot map
  attend   attention of one new token per request over its whole cache
  select   the blocks with the highest score bound for each request, and attention over them
"""
import math
import random

import torch

own = False

D, BLOCK, REC = 128, 64, 9216
SCALE2 = 1.4426950408889634 / math.sqrt(D)  # scores in base 2


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a serving loop: every request grows by a token, tables and slot map follow
        {"name": "index_decode_b64", "op": "index", "batch": 64, "ctx": 8192, "new": 1, "refill": False},
        # a batch of finished requests leaves and as many prompts of mixed lengths are admitted
        {"name": "index_refill_b512", "op": "index", "batch": 512, "ctx": 8192, "new": 8192, "refill": True},
        # one decode step's new keys and values of one layer, requests at any offset of their block
        {"name": "append_decode_b64_h16", "op": "append", "batch": 64, "ctx": 4096, "new": 1, "kv": 16},
        # chunks of prompts of mixed lengths entering the cache, from one token up
        {"name": "append_prefill_b8_h16", "op": "append", "batch": 8, "ctx": 4096, "new": 4096, "kv": 16},
        # one request's cached prefix handed back to a prefill attention
        {"name": "read_n4096_h16", "op": "read", "batch": 1, "ctx": 4096, "kv": 16},
        # the prefixes of several requests of mixed lengths
        {"name": "read_b6_n32768_h8", "op": "read", "batch": 6, "ctx": 32768, "kv": 8},
        # the smallest: one request just past its prompt, latency alone
        {"name": "attend_b1_n256_h16", "op": "attend", "batch": 1, "ctx": 256, "ragged": False, "kv": 16, "group": 1},
        # an ordinary mixed batch, one query head per key-value head
        {"name": "attend_b64_n8191_h16", "op": "attend", "batch": 64, "ctx": 8191, "ragged": True, "kv": 16, "group": 1},
        # the largest: long contexts, four query heads share a key-value head
        {"name": "attend_b16_n32768_h8x4", "op": "attend", "batch": 16, "ctx": 32768, "ragged": False, "kv": 8, "group": 4},
        # one long request, a tenth of its blocks
        {"name": "select_b1_n32768_h16", "op": "select", "batch": 1, "ctx": 32768, "ragged": False, "kv": 16, "group": 1, "keep": 52},
        # a mixed batch whose short requests keep every block they have
        {"name": "select_b64_n8191_h4x8", "op": "select", "batch": 64, "ctx": 8191, "ragged": True, "kv": 4, "group": 8, "keep": 16},
        # the long contexts again, a tenth of their blocks
        {"name": "select_b16_n32768_h8x4", "op": "select", "batch": 16, "ctx": 32768, "ragged": False, "kv": 8, "group": 4, "keep": 52},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["index", "append", "read", "attend", "select"])
    if op == "index":
        refill = rng.random() < 0.5
        return {"op": op, "batch": _spread(rng, 1, 512), "ctx": _spread(rng, 1, 8192), "new": _spread(rng, 1, 8192) if refill else 1, "refill": refill}
    kv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "append":
        new = 1 if rng.random() < 0.4 else _spread(rng, 1, 4096)
        return {"op": op, "batch": _spread(rng, 1, 64 if new == 1 else 8), "ctx": _spread(rng, 1, 4096), "new": new, "kv": kv}
    if op == "read":
        return {"op": op, "batch": _spread(rng, 1, 6), "ctx": _spread(rng, 1, 32768), "kv": min(kv, 8)}
    batch = _spread(rng, 1, 64)
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    ctx = _spread(rng, 1, max(64, min(32768, 16 * 32768 * 8 * 4 // (batch * kv * max(4, group)))))
    case = {"op": op, "batch": batch, "ctx": ctx, "ragged": rng.random() < 0.6, "kv": kv, "group": group}
    if op == "select":
        case["keep"] = _spread(rng, 1, 64)
    return case


def _mixed(n, most, salt):
    """n whole numbers in [1, most], spread over their logarithm, the first of them `most`: a part of the case, whatever the seed."""
    r = random.Random(1000003 * n + 10007 * most + salt)
    return [most] + [_spread(r, 1, most) for _ in range(n - 1)]


def _lengths(case):
    """Tokens that each request holds before the pass, and those that the pass adds."""
    b, op = case["batch"], case["op"]
    if op == "index":
        return _mixed(b, case["ctx"], 1), (_mixed(b, case["new"], 2) if case["new"] > 1 else [1] * b)
    if op == "append":
        r = random.Random(31 * b + case["ctx"])
        return [case["ctx"]] + [r.randint(0, case["ctx"]) for _ in range(b - 1)], (_mixed(b, case["new"], 3) if case["new"] > 1 else [1] * b)
    if op == "read" or case["ragged"]:
        return _mixed(b, case["ctx"], 4), [0] * b
    return [case["ctx"]] * b, [0] * b


def _full(n):
    """Blocks of a request of n tokens that are INT4 records (the last 1..64 tokens are in the tail)."""
    return (n - 1) // BLOCK if n > 0 else 0


def _touched(c, n):
    """First token of the blocks that an append of n tokens after c touches."""
    return BLOCK * _full(c)


# ---------------------------------------------------------------------------------------- prepare
def _random_records(count, kv, g, dev):
    """Records of `count` pages whose keys have channels of their own scale and mean, as rotated keys have, and a drift from block to block."""
    chan = torch.randn(1, kv, 1, D, generator=g, device=dev) * 0.5
    size = torch.exp(torch.randn(1, kv, 1, D, generator=g, device=dev) * 0.3)
    drift = torch.randn(count, kv, 1, D, generator=g, device=dev) * 0.3
    k = ((torch.randn(count, kv, BLOCK, D, generator=g, device=dev) + drift) * size + chan).bfloat16()
    v = torch.randn(count, kv, BLOCK, D, generator=g, device=dev).bfloat16()
    return _records(k.float(), v.float())


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(1000 + seed)
    b, op = case["batch"], case["op"]
    have, new = _lengths(case)
    order = torch.randperm(b, generator=g, device=dev)
    slots = order.to(torch.int32)  # the batch is in another order than the table's rows
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if op == "index":
        # room for hundreds of thousands of passes of one token each
        max_pages = 8192 if not case["refill"] else max(blocks(max(have)), blocks(max(new)), 1)
        pages = b * max_pages
    else:
        max_pages = max(blocks(h + n) for h, n in zip(have, new)) + 1
        pages = sum(blocks(h + n) for h, n in zip(have, new)) + 3
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    after = [h + (n if op == "append" else 0) for h, n in zip(have, new)]
    owned = torch.tensor([blocks(n) for n in after], device=dev)
    cols = torch.arange(max_pages, device=dev)
    first = torch.cumsum(owned, 0) - owned
    rows = torch.where(cols < owned[:, None], ids[(first[:, None] + cols).clamp(max=pages - 1)], -1)
    table = torch.full((b, max_pages), -1, dtype=torch.int32, device=dev)
    table[order] = rows.to(torch.int32)
    length = torch.zeros(b, dtype=torch.int32, device=dev)
    length[order] = torch.tensor(after, dtype=torch.int32, device=dev)
    used = sum(blocks(n) for n in after)
    free = torch.zeros(pages, dtype=torch.int32, device=dev)
    free[: pages - used] = ids[used:]
    s = {"case": dict(case), "slots": slots, "table": table, "length": length, "free": free,
         "n_free": torch.tensor([pages - used], dtype=torch.int32, device=dev),
         "n_new": torch.tensor(new, dtype=torch.int32, device=dev)}
    cu = lambda ns: torch.tensor([0] + torch.tensor(ns).cumsum(0).tolist(), dtype=torch.int32, device=dev)  # noqa: E731
    if op == "index":
        t = sum(new)
        s["tokens"] = t
        s["start"] = torch.empty(b, dtype=torch.int32, device=dev)
        s["cu"] = torch.empty(b + 1, dtype=torch.int32, device=dev)
        s["slot_map"] = torch.empty(t, dtype=torch.int32, device=dev)
        s["pos"] = torch.empty(t, dtype=torch.int32, device=dev)
        return s
    kv = case["kv"]
    s["rec"] = torch.empty(pages, kv, REC, dtype=torch.uint8, device=dev)
    step = max(1, 4096 // kv)
    for p in range(0, pages, step):
        n = min(step, pages - p)
        s["rec"][p: p + n] = _random_records(n, kv, g, dev)
    s["tail_k"] = torch.randn(b, kv, BLOCK, D, generator=g, device=dev).bfloat16()
    s["tail_v"] = torch.randn(b, kv, BLOCK, D, generator=g, device=dev).bfloat16()
    if op in ("append", "read"):
        # the tokens that come back: those of the blocks the append touches, or all of them
        begin = [_touched(h, n) if op == "append" else 0 for h, n in zip(have, new)]
        count = [a - f for a, f in zip(after, begin)]
        t = sum(count)
        s["slot_map"], _ = _places(slots, length, table, torch.tensor(begin, dtype=torch.int32, device=dev), cu(count), t, pages)
        s["out_k"] = torch.empty(t, kv, D, dtype=torch.bfloat16, device=dev)
        s["out_v"] = torch.empty(t, kv, D, dtype=torch.bfloat16, device=dev)
    if op == "append":
        t = sum(new)
        s["start"] = torch.tensor(have, dtype=torch.int32, device=dev)
        s["cu"] = cu(new)
        s["k"] = (torch.randn(t, kv, D, generator=g, device=dev) + 0.5).bfloat16()
        s["v"] = torch.randn(t, kv, D, generator=g, device=dev).bfloat16()
        s["items"] = sum(_full(a) - _full(h) for a, h in zip(after, have))
    if op in ("attend", "select"):
        heads = kv * case["group"]
        s["q"] = (torch.randn(b, heads, D, generator=g, device=dev) * 1.5).bfloat16()
        s["o"] = torch.empty(b, heads, D, dtype=torch.float32, device=dev)
        s["lse"] = torch.empty(b, heads, dtype=torch.float32, device=dev)
        if op == "select":
            s["sel"] = torch.empty(b, kv, case["keep"], dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _group(x, dim):
    """Codes, scale and zero of 4-bit groups along `dim`: the scale and zero are rounded to 16 bits first, the codes taken against those."""
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s, z = ((hi - lo) / 15.0).half().float(), lo.half().float()
    codes = torch.where(s == 0, torch.zeros_like(x), torch.round((x - z) / torch.where(s == 0, torch.ones_like(s), s)).clamp(0, 15))
    return codes.to(torch.uint8), s.half(), z.half()


def _records(k, v):
    """Keys and values [n][kv][64][128] as group records [n][kv][9216]: keys in groups of a channel, values in groups of half a token."""
    n, kv = k.shape[:2]
    kc, ks, kz = _group(k, 2)
    vc, vs, vz = _group(v.view(n, kv, BLOCK, 2, D // 2), 4)
    vc = vc.view(n, kv, BLOCK, D)
    codes = torch.cat([kc[..., 0::2] | kc[..., 1::2] << 4, vc[..., 0::2] | vc[..., 1::2] << 4], -1).reshape(n, kv, BLOCK * D)
    vsz = torch.cat([vs, vz], -1).view(n, kv, BLOCK * 4).view(torch.uint8)
    ksz = torch.stack([ks, kz], -1).view(n, kv, D * 2).view(torch.uint8)
    return torch.cat([codes, vsz, ksz], -1)


def _values(rec):
    """Keys and values [..][64][128] in 32 bits of group records [..][9216]."""
    lead = rec.shape[:-1]
    codes = rec[..., : BLOCK * D].reshape(*lead, BLOCK, 2, D // 2)
    codes = torch.stack([codes & 15, codes >> 4], -1).reshape(*lead, BLOCK, 2, D).float()
    vsz = rec[..., BLOCK * D: BLOCK * D + 512].contiguous().view(torch.float16).reshape(*lead, BLOCK, 2, 1, 2).float()
    ksz = rec[..., BLOCK * D + 512:].contiguous().view(torch.float16).reshape(*lead, 1, D, 2).float()
    k = codes[..., 0, :] * ksz[..., 0] + ksz[..., 1]
    v = (codes[..., 1, :].reshape(*lead, BLOCK, 2, D // 2) * vsz[..., 0] + vsz[..., 1]).reshape(*lead, BLOCK, D)
    return k, v


def _places(slots, length, table, start, cu, tokens, pages):
    """The place and position of every token: page * 64 + offset, or behind all pages the tail's rows."""
    t = torch.arange(tokens, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True).clamp(max=len(slots) - 1)
    pos = start[b] + (t - cu[b])
    slot, block = slots[b].long(), pos // BLOCK
    full = ((length[slot] - 1).clamp(min=0)) // BLOCK
    page = table[slot, block.long().clamp(max=table.shape[1] - 1)]
    place = torch.where(block < full, page, (pages + slot).to(torch.int32)) * BLOCK + pos % BLOCK
    return place.to(torch.int32), pos.to(torch.int32)


def _plain_release(s):
    slots, length, table, free, n_free = s["slots"].long(), s["length"], s["table"], s["free"], s["n_free"]
    owned = (length[slots] + BLOCK - 1) // BLOCK
    before = torch.cumsum(owned, 0) - owned
    cols = torch.arange(table.shape[1], device=table.device)
    to = torch.where(cols < owned[:, None], n_free + before[:, None] + cols, free.numel())
    longer = torch.cat([free, free[:1]])
    longer.scatter_(0, to.reshape(-1), table[slots].reshape(-1))
    free.copy_(longer[:-1])
    n_free += owned.sum().to(torch.int32)
    table[slots] = -1
    length[slots] = 0


def _plain_extend(s):
    slots, length, table, free, n_free, new = s["slots"].long(), s["length"], s["table"], s["free"], s["n_free"], s["n_new"]
    have = length[slots]
    first = (have + BLOCK - 1) // BLOCK
    need = (have + new + BLOCK - 1) // BLOCK - first
    upto = torch.cumsum(need, 0)
    rel = torch.arange(table.shape[1], device=table.device) - first[:, None]
    pick = (n_free - 1 - (upto - need)[:, None] - rel).clamp(0, free.numel() - 1)
    table[slots] = torch.where((rel >= 0) & (rel < need[:, None]), free[pick.long()], table[slots])
    length[slots] = have + new
    n_free -= upto[-1].to(torch.int32)
    s["start"].copy_(have)
    s["cu"].copy_(torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0).to(torch.int32)]))
    place, pos = _places(s["slots"], length, table, s["start"], s["cu"], s["tokens"], free.numel())
    s["slot_map"].copy_(place)
    s["pos"].copy_(pos)


def _plain_append(s):
    slots, start, cu, table = s["slots"].long(), s["start"].long(), s["cu"].long(), s["table"]
    count = cu[1:] - cu[:-1]
    after = start + count
    full0, full1 = (start - 1).clamp(min=0) // BLOCK, (after - 1).clamp(min=0) // BLOCK
    dev = slots.device
    i64 = torch.arange(BLOCK, device=dev)
    if s["items"]:
        # the blocks that fill up: row i of block p is token 64 p + i, old ones in the tail, new ones in the input
        done = full1 - full0
        b = torch.repeat_interleave(torch.arange(len(slots), device=dev), done, output_size=s["items"])
        block = full0[b] + torch.arange(s["items"], device=dev) - (torch.cumsum(done, 0) - done)[b]
        token = block[:, None] * BLOCK + i64
        old = (token < start[b, None])[..., None, None]
        row = (cu[b, None] + token - start[b, None]).clamp(0, s["k"].shape[0] - 1)
        k = torch.where(old, s["tail_k"][slots[b]].transpose(1, 2), s["k"][row])
        v = torch.where(old, s["tail_v"][slots[b]].transpose(1, 2), s["v"][row])
        s["rec"][table[slots[b], block].long()] = _records(k.transpose(1, 2).float(), v.transpose(1, 2).float())
    # the rows of the last block
    token = full1[:, None] * BLOCK + i64
    mine = ((token >= start[:, None]) & (token < after[:, None]))[:, None, :, None]
    row = (cu[:-1, None] + token - start[:, None]).clamp(0, s["k"].shape[0] - 1)
    s["tail_k"][slots] = torch.where(mine, s["k"][row].transpose(1, 2), s["tail_k"][slots])
    s["tail_v"][slots] = torch.where(mine, s["v"][row].transpose(1, 2), s["tail_v"][slots])


def _plain_read(s):
    place = s["slot_map"].long()
    pages = s["rec"].shape[0]
    page, i = place // BLOCK, place % BLOCK
    in_tail = (page >= pages)[:, None, None]
    at, slot = page.clamp(max=pages - 1), (page - pages).clamp(min=0)
    kv = s["rec"].shape[1]
    codes = s["rec"][:, :, : BLOCK * D].view(pages, kv, BLOCK, D)[at, :, i]
    codes = torch.stack([codes & 15, codes >> 4], -1).view(len(place), kv, 2, D).float()
    vsz = s["rec"][:, :, BLOCK * D: BLOCK * D + 512].unflatten(2, (BLOCK, 8))[at, :, i].contiguous().view(torch.float16).view(-1, kv, 2, 1, 2).float()
    ksz = s["rec"][:, :, BLOCK * D + 512:][at].contiguous().view(torch.float16).view(-1, kv, D, 2).float()
    k = codes[:, :, 0] * ksz[..., 0] + ksz[..., 1]
    v = (codes[:, :, 1].view(-1, kv, 2, D // 2) * vsz[..., 0] + vsz[..., 1]).view(-1, kv, D)
    s["out_k"].copy_(torch.where(in_tail, s["tail_k"][slot, :, i].float(), k))
    s["out_v"].copy_(torch.where(in_tail, s["tail_v"][slot, :, i].float(), v))


def _plain_select(s):
    """The blocks of the highest bounds: score(block) = max over the group's queries of sum_c max(q_c lo_c, q_c hi_c)."""
    case, slots = s["case"], s["slots"].long()
    kv, group, keep = case["kv"], case["group"], case["keep"]
    full = (s["length"][slots] - 1).clamp(min=0) // BLOCK
    most = s["table"].shape[1]
    pages = s["table"][slots].long().clamp(min=0)
    ksz = s["rec"][:, :, BLOCK * D + 512:][pages].contiguous().view(torch.float16).view(len(slots), most, kv, D, 2).double()
    lo, hi = ksz[..., 1], ksz[..., 1] + 15.0 * ksz[..., 0]
    q = s["q"].view(len(slots), kv, group, D).double()
    score = torch.matmul(q.clamp(min=0), hi.permute(0, 2, 3, 1)) + torch.matmul(q.clamp(max=0), lo.permute(0, 2, 3, 1))
    score = score.amax(2)
    there = (torch.arange(most, device=slots.device) < full[:, None])[:, None]
    order = torch.sort(torch.where(there, score, -math.inf), dim=-1, descending=True, stable=True).indices
    order = torch.nn.functional.pad(order[..., :keep], (0, max(0, keep - most)), value=most)
    taken = torch.where(torch.arange(keep, device=slots.device) < full[:, None, None], order, most)
    taken = torch.sort(taken, dim=-1).values
    s["sel"].copy_(torch.where(taken < full[:, None, None], taken, -1))


def _plain_attend(s, sel=None):
    case, slots = s["case"], s["slots"].long()
    n, kv, group = len(slots), case["kv"], case["group"]
    length = s["length"][slots].long()
    full = (length - 1).clamp(min=0) // BLOCK
    if sel is None:
        blocks = torch.arange(s["table"].shape[1], device=slots.device).expand(n, kv, -1)
    else:
        blocks = sel.long()
    there = (blocks >= 0) & (blocks < full[:, None, None])
    page = s["table"][slots[:, None, None], blocks.clamp(min=0)].long().clamp(min=0)
    k, v = _values(s["rec"][page, torch.arange(kv, device=slots.device)[:, None]])  # [n][kv][blocks][64][128]
    q = s["q"].view(n, kv, group, D).float()
    tk, tv = s["tail_k"][slots].float(), s["tail_v"][slots].float()
    in_tail = (torch.arange(BLOCK, device=slots.device) < (length - BLOCK * full)[:, None])[:, None, :, None]
    tk, tv = torch.where(in_tail, tk, 0.0), torch.where(in_tail, tv, 0.0)
    x = torch.cat([torch.matmul(q, k.flatten(2, 3).transpose(2, 3)), torch.matmul(q, tk.transpose(2, 3))], -1) * SCALE2
    ok = torch.cat([there.repeat_interleave(BLOCK, 2), in_tail[..., 0].expand(n, kv, BLOCK)], 2)[:, :, None]
    x = torch.where(ok, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.where(ok, torch.exp2(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = p.sum(-1, keepdim=True)
    m = k.shape[2] * BLOCK
    o = torch.matmul(p[..., :m], v.flatten(2, 3)) + torch.matmul(p[..., m:], tv)
    s["o"].copy_((o / torch.where(total == 0, 1.0, total)).view(n, kv * group, D))
    s["lse"].copy_((top + torch.log2(total)).view(n, kv * group))


# -------------------------------------------------------------------------------------------- run
def _handles(s):
    """What a serving program makes once and keeps: the index, the pool and the workspace."""
    from quantized_kv_attention_int4_b200 import paged
    if "index" not in s:
        s["index"] = paged.PagedIndex(s["table"], s["length"], s["free"], s["n_free"])
        if "rec" in s:
            s["pool"] = paged.PagedPool(s["rec"], s["tail_k"], s["tail_v"])
        if "q" in s:
            s["ws"] = paged.workspace(s["index"], s["pool"], s["q"].shape[0], s["q"].shape[1])
    return paged


def run(s):
    op = s["case"]["op"]
    if op == "index":
        if own:
            paged = _handles(s)
            if s["case"]["refill"]:
                paged.fl_paged_release(s["index"], s["slots"])
            paged.fl_paged_extend(s["index"], s["slots"], s["n_new"], s["start"], s["cu"])
            paged.fl_paged_slot_map(s["index"], s["slots"], s["start"], s["cu"], s["slot_map"], s["pos"])
        else:
            if s["case"]["refill"]:
                _plain_release(s)
            _plain_extend(s)
        return [s["table"], s["length"], s["free"], s["n_free"], s["start"], s["cu"], s["slot_map"], s["pos"]]
    if op == "append":
        # the records are 4-bit codes: they come back as the values they stand for, through a read of the touched blocks
        if own:
            paged = _handles(s)
            paged.fl_paged_append(s["index"], s["pool"], s["slots"], s["start"], s["cu"], s["k"], s["v"])
            paged.fl_paged_read(s["index"], s["pool"], s["slot_map"], s["out_k"], s["out_v"])
        else:
            _plain_append(s)
            _plain_read(s)
        return [s["out_k"], s["out_v"], s["tail_k"], s["tail_v"]]
    if op == "read":
        if own:
            paged = _handles(s)
            paged.fl_paged_read(s["index"], s["pool"], s["slot_map"], s["out_k"], s["out_v"])
        else:
            _plain_read(s)
        return [s["out_k"], s["out_v"]]
    if op == "attend":
        if own:
            paged = _handles(s)
            paged.fl_paged_attn_decode(s["index"], s["pool"], s["slots"], s["q"], s["o"], s["ws"], lse=s["lse"])
        else:
            _plain_attend(s)
        return [s["o"], s["lse"]]
    if own:
        paged = _handles(s)
        paged.fl_paged_select(s["index"], s["pool"], s["slots"], s["q"], s["sel"], s["ws"])
        paged.fl_paged_attn_decode(s["index"], s["pool"], s["slots"], s["q"], s["o"], s["ws"], lse=s["lse"], sel=s["sel"])
    else:
        _plain_select(s)
        _plain_attend(s, s["sel"])
    return [s["sel"], s["o"], s["lse"]]


def work(case):
    have, new = _lengths(case)
    op, b = case["op"], case["batch"]
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if op == "index":
        base = [0] * b if case["refill"] else have
        taken = sum(blocks(h + n) - blocks(h) for h, n in zip(base, new))
        given = sum(blocks(h) for h in have) if case["refill"] else 0
        # slots, new counts, lengths in and out, starts and offsets; a page id in and out; a place and a position
        return {"bytes": 24 * b + 4 + 8 * taken + 12 * given + 8 * sum(new), "flops": 0}
    kv = case["kv"]
    token = 4 * D * kv  # bytes of a token's BF16 keys and values
    if op == "append":
        full = sum(_full(h + n) - _full(h) for h, n in zip(have, new))
        old = sum(min(h, BLOCK * _full(h + n)) - BLOCK * _full(h) for h, n in zip(have, new) if _full(h + n) > _full(h))
        tail = sum(min(n, h + n - BLOCK * _full(h + n)) for h, n in zip(have, new))
        back = sum(h + n - _touched(h, n) for h, n in zip(have, new))
        in_tail = sum(h + n - BLOCK * _full(h + n) for h, n in zip(have, new))
        return {"bytes": token * (sum(new) + old + tail + back + in_tail) + full * kv * REC * 2 + 4 * back, "flops": 0}
    if op == "read":
        full = sum(_full(h) for h in have)
        return {"bytes": token * (2 * sum(have) - BLOCK * full) + full * kv * REC + 4 * sum(have), "flops": 0}
    group = case["group"]
    full = [_full(h) for h in have]
    tails = sum(h - BLOCK * f for h, f in zip(have, full))
    io = b * kv * group * D * 6 + b * kv * group * 4
    seen, scored, extra = sum(full), 0, 0
    if op == "select":
        keep = case["keep"]
        seen, scored = sum(min(f, keep) for f in full), sum(f for f in full if f > keep)
        extra = sum(f - keep for f in full if f > keep)  # a block that is scored and then attended to is read once
        io += 4 * b * kv * keep
    return {"bytes": seen * kv * REC + extra * kv * D * 4 + tails * token + io + 4 * sum(full),
            "flops": 4 * D * group * kv * (seen * BLOCK + tails) + 2 * D * group * kv * scored}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The same from the definitions, request by request, in 64 bits; a group's scale, zero and codes are rounded as the cache's format says."""
    op = case["op"]
    if op == "index":
        return None  # whole numbers alone
    s = prepare(case, seed)
    slots, length = s["slots"].tolist(), s["length"].tolist()
    pages, kv = s["rec"].shape[0], case["kv"]

    def unpack(rec):  # [m][9216] -> keys, values [m][64][128] in 64 bits
        m = rec.shape[0]
        halves = rec[:, BLOCK * D:].contiguous().view(torch.float16).double()
        c = rec[:, : BLOCK * D].reshape(m, BLOCK, 2, D // 2).to(torch.int16)
        out = torch.empty(m, 2, BLOCK, D, dtype=torch.float64, device=rec.device)
        out[..., 0::2] = (c % 16).double().transpose(1, 2)
        out[..., 1::2] = (c // 16).double().transpose(1, 2)
        vs, ks = halves[:, : BLOCK * 4].reshape(m, BLOCK, 2, 2), halves[:, BLOCK * 4:].reshape(m, D, 2)
        k = out[:, 0] * ks[:, None, :, 0] + ks[:, None, :, 1]
        v = out[:, 1] * vs[..., 0].repeat_interleave(D // 2, 2) + vs[..., 1].repeat_interleave(D // 2, 2)
        return k, v

    def rounded(x):  # groups along the last axis, through the 4-bit format; every step in 64 bits, then to the step's own type
        f32 = lambda y: y.float().double()  # noqa: E731
        lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        sc, z = f32(f32(hi - lo) / 15.0).half().double(), lo.half().double()
        code = torch.round(f32(f32(x - z) / sc)).clamp(0, 15)
        return torch.where(sc == 0, z, code * sc + z)

    if op in ("append", "read"):
        outs = []
        if op == "append":
            start, cu = s["start"].tolist(), s["cu"].tolist()
            new_k, new_v = s["tail_k"].double(), s["tail_v"].double()
        for i, slot in enumerate(slots):
            n = length[slot]
            f = _full(n)
            if op == "read":
                ks, vs = [], []
                if f:
                    rec = s["rec"][s["table"][slot, :f].long()]
                    k, v = unpack(rec.reshape(f * kv, REC))
                    ks.append(k.reshape(f, kv, BLOCK, D).transpose(1, 2).reshape(f * BLOCK, kv, D))
                    vs.append(v.reshape(f, kv, BLOCK, D).transpose(1, 2).reshape(f * BLOCK, kv, D))
                ks.append(s["tail_k"][slot, :, : n - BLOCK * f].double().transpose(0, 1))
                vs.append(s["tail_v"][slot, :, : n - BLOCK * f].double().transpose(0, 1))
                outs.append((torch.cat(ks), torch.cat(vs)))
                continue
            c = start[i]
            base = BLOCK * _full(c)
            k = torch.cat([s["tail_k"][slot, :, : c - base].double().transpose(0, 1), s["k"][cu[i]: cu[i + 1]].double()])
            v = torch.cat([s["tail_v"][slot, :, : c - base].double().transpose(0, 1), s["v"][cu[i]: cu[i + 1]].double()])
            whole = BLOCK * f - base
            new_k[slot, :, max(0, c - BLOCK * f): n - BLOCK * f] = k[whole + max(0, c - BLOCK * f):].transpose(0, 1)
            new_v[slot, :, max(0, c - BLOCK * f): n - BLOCK * f] = v[whole + max(0, c - BLOCK * f):].transpose(0, 1)
            if whole:
                k[:whole] = rounded(k[:whole].reshape(-1, BLOCK, kv, D).permute(0, 2, 3, 1)).permute(0, 3, 1, 2).reshape(whole, kv, D)
                v[:whole] = rounded(v[:whole].reshape(whole, kv, 2, D // 2)).reshape(whole, kv, D)
            outs.append((k, v))
        out = [torch.cat([k for k, _ in outs]), torch.cat([v for _, v in outs])]
        return out + [new_k, new_v] if op == "append" else out
    group = case["group"]
    o = torch.zeros(len(slots), kv * group, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((len(slots), kv * group), -math.inf, dtype=torch.float64, device=o.device)
    for i, slot in enumerate(slots):
        n = length[slot]
        f = _full(n)
        for h in range(kv):
            q = s["q"][i, h * group: (h + 1) * group].double()
            page = s["table"][slot, :f].long()
            if op == "select" and f > case["keep"]:
                sz = s["rec"][page, h, BLOCK * D + 512:].contiguous().view(torch.float16).double().reshape(f, 1, D, 2)
                bound = torch.maximum(q * sz[..., 1], q * (sz[..., 1] + 15 * sz[..., 0])).sum(-1).max(1).values
                best = sorted(range(f), key=lambda j, u=bound.tolist(): (-u[j], j))[: case["keep"]]
                page = page[torch.tensor(sorted(best), device=page.device)]
            k, v = unpack(s["rec"][page, h])
            k = torch.cat([k.reshape(-1, D), s["tail_k"][slot, h, : n - BLOCK * f].double()])
            v = torch.cat([v.reshape(-1, D), s["tail_v"][slot, h, : n - BLOCK * f].double()])
            x = q @ k.T / math.sqrt(D)
            o[i, h * group: (h + 1) * group] = torch.softmax(x, -1) @ v
            lse[i, h * group: (h + 1) * group] = torch.logsumexp(x, -1) / math.log(2.0)
    return [None, o, lse] if op == "select" else [o, lse]
