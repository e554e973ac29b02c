"""The paged cache on the GPU at the edges of what its header allows: wrong counts, damaged
tables, the largest batches, wide tables, and the kernels that only large calls take."""
import numpy as np
import pytest
import torch

from oracle.paged_oracle import PAGE
from pagedhelpers import Pair, i32
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
