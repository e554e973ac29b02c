"""The paged oracle against hand-made states and, block by block, against the single-sequence
oracle's codec and attention."""
import numpy as np

from oracle import flashloop_oracle as fo
from oracle.paged_oracle import D, PAGE, PagedOracle, blocks, full, record, unrecord


def test_blocks_of_a_request():
    assert [full(n) for n in (0, 1, 63, 64, 65, 128, 129)] == [0, 0, 0, 0, 1, 1, 2]
    assert [blocks(n) for n in (0, 1, 64, 65, 128, 129)] == [0, 1, 1, 2, 2, 3]


def test_pages_are_taken_and_given_back_in_order():
    o = PagedOracle(3, 4, 6, 1)
    start, cu = o.extend([2, 0], [65, 1])
    assert start.tolist() == [0, 0] and cu.tolist() == [0, 65, 66]
    assert o.table[2, :2].tolist() == [0, 1] and o.table[0, 0] == 2 and o.free == [5, 4, 3]
    start, cu = o.extend([0, 1, 2, -1, 0], [63, 256, 10, 7, 1])   # the second needs 4 of the 3 free pages
    assert start.tolist() == [1, -1, 65, -1, -1] and cu.tolist() == [0, 63, 319, 329, 336, 337]
    assert o.errors == [(18, 1), (17, 4)] and o.length.tolist() == [64, 0, 75]
    place, pos = o.slot_map([2], [60], [0, 8], 9)
    assert pos.tolist() == [60, 61, 62, 63, 64, 65, 66, 67, -7]
    assert place.tolist() == [60, 61, 62, 63] + [(6 + 2) * 64 + i for i in range(4)] + [-7]
    o.release([2, 1], 2)
    assert o.free == [5, 4, 3, 0, 1] and o.length.tolist() == [64, 0, 0]


def test_records_are_the_codec_of_the_single_sequence_cache():
    r = np.random.default_rng(0)
    k, v = r.standard_normal((2, PAGE, D)).astype(np.float32)
    kh, vh = fo.decode_base(fo.encode_base(k[None], v[None]))
    ku, vu, sz = unrecord(record(k, v))
    assert np.array_equal(ku.astype(np.float32), kh[0]) and np.array_equal(vu.astype(np.float32), vh[0])
    assert np.all(ku <= sz[:, 1] + 15 * sz[:, 0]) and np.all(ku >= sz[:, 1])


def test_append_in_pieces_equals_append_at_once():
    r = np.random.default_rng(1)
    n = 200
    k, v = r.standard_normal((2, n, 2, D)).astype(np.float32)
    one, many = PagedOracle(1, 4, 4, 2), PagedOracle(1, 4, 4, 2)
    s, cu = one.extend([0], [n])
    one.append([0], s, cu, k, v)
    at = 0
    for m in (1, 62, 1, 1, 64, 65, 6):
        s, cu = many.extend([0], [m])
        many.append([0], s, cu, k[at: at + m], v[at: at + m])
        at += m
    assert at == n and np.array_equal(one.rec, many.rec)
    assert np.array_equal(one.tail[:, 0, :, :8], many.tail[:, 0, :, :8])
    q = r.standard_normal((3, D))
    kk, vv = one.keys_values(0, 1)
    ref = np.stack([fo.attention_dense(q[i][None], kk[None], vv[None])[0][0] for i in range(3)])
    np.testing.assert_allclose(one.attend(0, 1, q)[0], ref, rtol=1e-12, atol=1e-13)


def test_scores_bound_every_key_of_their_block():
    r = np.random.default_rng(2)
    o = PagedOracle(1, 8, 8, 1)
    s, cu = o.extend([0], [8 * 64])
    k = (r.standard_normal((512, 1, D)) + np.repeat(r.standard_normal((8, 1, D)), 64, 0)).astype(np.float32)
    o.append([0], s, cu, k, k)
    q = r.standard_normal((2, D))
    best = o.select(0, 0, q, 1)[0]
    bounds = []
    for j in range(7):
        kh, _, sz = unrecord(o.rec[o.table[0, j], 0])
        b = np.maximum(q * sz[:, 1], q * (sz[:, 1] + 15 * sz[:, 0])).sum(-1).max()
        assert b >= (q @ kh.T).max()
        bounds.append(b)
    assert best == int(np.argmax(bounds))
    assert o.select(0, 0, q, 7) == list(range(7))
