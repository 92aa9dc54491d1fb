"""Pins of the oracle of the speculative-decoding operators: hand-written tables and trees, agreement
of the tree attention with the decode-attention oracle (one node; a chain as decode steps of growing
length), facts of the definition, and the sequential move of accepted rows."""
import numpy as np

import oracle
from oracle import speculative as spec


def _codes(shape, rng, hi=0x70):
    c = rng.integers(0x08, hi, size=shape).astype(np.uint8)
    return c | (rng.integers(0, 2, size=shape).astype(np.uint8) << 7)


def test_codec_agrees_with_the_c_oracle():
    np.testing.assert_array_equal(spec.e4m3_values(), oracle.e4m3_decode_all())


def test_tables_by_hand():
    table = [[4, -1, -1], [-1, -1, -1], [7, 2, -1]]
    t, cu, lens, slots, pos, left = spec.batch_tables(
        [3, 0, 8], [3, 0, 2], table, 4, [9, 5, 6, 1], 3, 7)
    assert t.tolist() == [[4, 6, -1], [-1, -1, -1], [7, 2, 5]]
    assert cu.tolist() == [0, 3, 3, 5] and lens.tolist() == [6, 0, 10] and left == 1
    assert slots.tolist() == [19, 24, 25, 20, 21, -1, -1]
    assert pos.tolist() == [3, 4, 5, 8, 9, 0, 0]


def test_tree_by_hand():
    #  -1 -> 0 -> 1 -> 3;  0 -> 2;  -1 -> 4
    sees = spec.tree_sees([-1, 0, 0, 1, -1])
    assert spec.pack_bits(sees, 1)[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000]
    chain = spec.tree_sees(np.arange(-1, 69))
    bits = spec.pack_bits(chain, 2).view(np.uint64)
    assert bits[63].tolist() == [2 ** 64 - 1, 0] and bits[69].tolist() == [2 ** 64 - 1, 63]


def test_one_node_and_chains_are_decode_steps():
    rng = np.random.default_rng(3)
    Hq, Hkv, D, bs = 4, 2, 32, 4
    k, v = _codes((64, Hkv * D), rng), _codes((64, Hkv * D), rng)
    table = rng.permutation(16).reshape(2, 8).astype(np.int32)
    q = [_codes((3, Hq * D), rng, 0x38), _codes((5, Hq * D), rng, 0x38)]
    ctx, s3 = [0, 11], np.array([0.25, 0.125, 2.0], np.float32)
    chain = [np.tril(np.ones((len(x), len(x)), bool)) for x in q]
    out, absref, zabs, count = spec.attention(q, k, v, s3, table, ctx, chain, Hq, Hkv, bs)
    for i in range(5):
        rows = np.stack([q[0][min(i, 2)], q[1][i]])
        lens = np.array([min(i, 2) + 1, 11 + i + 1], np.int32)
        ref, aref, zref = oracle.attention_decode(rows, k, v, s3, table, lens, Hq, Hkv, D, bs)
        for b, node in ((0, min(i, 2)), (1, i)):
            np.testing.assert_allclose(out[b][node], ref[b], rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(absref[b][node], aref[b], rtol=1e-12)
            np.testing.assert_allclose(zabs[b][node], zref[b], rtol=1e-12)
            assert count[b][node] == lens[b]


def test_unseen_positions_do_not_count():
    rng = np.random.default_rng(4)
    k, v = _codes((32, 32), rng), _codes((32, 32), rng)
    table = np.array([[1, 3, 0, 2]], np.int32)
    q = [_codes((3, 32), rng, 0x38)]
    sees = [np.array([[0, 1, 1], [1, 0, 1], [0, 0, 0]], bool)]        # above the diagonal: ignored
    out, _, _, count = spec.attention(q, k, v, [1, 1, 1], table, [0], sees, 1, 1, 8)
    assert count[0].tolist() == [0, 1, 0]
    assert not out[0][0].any() and not out[0][2].any()
    np.testing.assert_array_equal(out[0][1], spec.e4m3_values()[v[8]])


def test_accept_by_hand():
    k = np.arange(24, dtype=np.uint8).reshape(12, 2)
    (got,), lens = spec.accept([k], [[2, 0]], [1], [[0, 1, 3]], [3], 4)
    # slots of positions 1.. are 9, 10, 11, 0, 1; node 3 (slot 0) moves to slot 11
    want = k.copy()
    want[11] = k[0]
    np.testing.assert_array_equal(got, want)
    assert lens.tolist() == [4]


def test_batch_tables_with_blocks_held():
    """By hand, blocks of 4: request 0 holds its context's block and one behind it (two of its tokens
    need a third), request 1 holds more than it needs, request 2 meets the end of the stack and holds
    only what it got."""
    table = [[3, 5, -1], [6, 7, 9], [0, -1, -1]]
    got = spec.batch_tables([4, 1, 4], [6, 2, 8], table, 4, [8, 2], 2, 16, held=[2, 3, 0])
    assert got[0].tolist() == [[3, 5, 2], [6, 7, 9], [0, 8, -1]]
    assert got[3].tolist() == [20, 21, 22, 23, 8, 9, 25, 26, 32, 33, 34, 35, -1, -1, -1, -1]
    assert got[5] == 0 and got[6].tolist() == [3, 3, 2]
