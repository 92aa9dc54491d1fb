"""GPU parity of the attention of drafted trees over the FP8 KV cache (fp8q_attention_tree) against the
float64 oracle: head layouts with 1 to 40 query heads per kv head, head sizes 64 and 128, ragged
drafts from no node to 1024, contexts from none to long, block sizes 1 to 128, arbitrary masks (rows
that see nothing among them), NaN codes in places that are not seen, scores that grow along the
positions, strided and padded rows, caches beyond 2^31 bytes, inputs out of range, captured and
replayed calls, and a whole speculative step.

The gate is the one of the decode attention, from the kernel's arithmetic: a score is a sum of D exact
products in fp32 then one scale, |dz| <= (D + 2) 2^-24 zabs, which moves a weight by at most 2 |dz|
relatively; a weight enters the value sum as fp16 (at most 2^-11 relatively); value sums, softmax sums,
merges and exp2 add at most (L + 16) 2^-23 of absref; the bf16 rounding half an ulp.  Weights far below
the largest one are fp16 subnormals: the largest weight is held between 2^7 and 2^15, a subnormal is
off by at most 2^-25, so each position adds at most 2^-32 of the largest value in magnitude:
    |out - ref| <= ulp_bf16(|ref|) / 2 + L 2^-32 vmax
                   + absref * (2^-11 + 2 (D + 2) 2^-24 zabs + (L + 16) 2^-23).
"""
import numpy as np
import pytest
import torch

import oracle
import fp8_blockwise_w8a8_b200 as fq
from oracle import speculative as spec

from helpers import host_bf16_f64

pytestmark = pytest.mark.gpu
RANGE = 9


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _codes(shape, rng, std=40.0):
    """E4M3 codes of N(0, std) values, as the cache holds them under a per-tensor scale."""
    x = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(std))
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _case(Hq, Hkv, D, nodes, ctx, bs, seed, kind="tree", spare=3):
    """Random codes, a shuffled block table and trees; kind "random" gives arbitrary masks."""
    rng = np.random.default_rng(seed)
    need = [-(-(c + n) // bs) for c, n in zip(ctx, nodes)]
    width = max(1, max(need))
    blocks = sum(need) + spare
    perm = rng.permutation(blocks)
    table = np.full((len(nodes), width), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    sees = []
    for n in nodes:
        if kind == "random":
            sees.append(rng.random((n, n)) < 0.4)
        elif kind == "chain":
            sees.append(np.tril(np.ones((n, n), bool)))
        else:
            sees.append(spec.tree_sees([rng.integers(max(-1, i - 5), i) for i in range(n)]))
    return dict(Hq=Hq, Hkv=Hkv, D=D, bs=bs, ctx=np.array(ctx), nodes=list(nodes), table=table,
                sees=sees, q=[_codes((n, Hq * D), rng) for n in nodes],
                k=_codes((blocks * bs, Hkv * D), rng), v=_codes((blocks * bs, Hkv * D), rng),
                s3=np.array([0.011, 0.012, 0.007], np.float32),
                max_nodes=max(1, max(nodes)), max_len=max(1, max(c + n for c, n in zip(ctx, nodes))))


def _args(d, mask=True):
    words = -(-d["max_nodes"] // 64)
    bits = np.concatenate([spec.pack_bits(s, words) for s in d["sees"]])
    return [dev(np.concatenate(d["q"])), dev(d["k"]), dev(d["v"]), dev(d["s3"]), i32(d["table"]),
            i32(d["ctx"]), i32(np.concatenate([[0], np.cumsum(d["nodes"])])),
            dev(bits) if mask else None, d["Hq"], d["Hkv"], d["bs"], d["max_nodes"], d["max_len"]]


def _oracle(d, sm_scale=None):
    return spec.attention(d["q"], d["k"], d["v"], d["s3"], d["table"], d["ctx"], d["sees"], d["Hq"],
                          d["Hkv"], d["bs"], sm_scale)


def _check(o, d, sm_scale=None, seqs=None):
    D = d["D"]
    got = host_bf16_f64(o)
    ref, absref, zabs, count = _oracle(d, sm_scale)
    cu = np.concatenate([[0], np.cumsum(d["nodes"])])
    vmax = float(d["s3"][2]) * 448.0
    for b in range(len(ref)) if seqs is None else seqs:
        L = count[b].astype(np.float64)[:, None]
        z = np.repeat(zabs[b], D, axis=1)
        bound = (oracle.bf16_ulp(np.abs(ref[b])) / 2 + L * 2.0 ** -32 * vmax
                 + absref[b] * (2.0 ** -11 + 2 * (D + 2) * 2.0 ** -24 * z + (L + 16) * 2.0 ** -23))
        err = np.abs(got[cu[b]:cu[b + 1]] - ref[b])
        bad = ~(err <= bound)
        assert not bad.any(), (f"sequence {b}: {bad.sum()} of {bad.size} outside the bound, first at "
                               f"{np.argwhere(bad)[0]}; largest excess {np.nanmax(err - bound):.3e}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (6, 2), (5, 1), (8, 2), (16, 2), (40, 1)])
def test_head_layouts_and_ragged_lengths(Hq, Hkv, D):
    d = _case(Hq, Hkv, D, [1, 3, 0, 17, 33, 64, 65, 2, 7], [0, 1, 40, 63, 64, 65, 127, 300, 0], 16,
              seed=Hq + Hkv + D)
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("bs", [1, 7, 64, 128])
def test_block_sizes(bs):
    d = _case(8, 2, 128, [5, 1, 12], [130, 77, 3], bs, seed=30 + bs)
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [1, 2, 3, 4, 6, 8, 12, 20, 24, 48, 64, 96, 100, 128, 640])
def test_block_sizes_on_both_sides_of_the_row_copies(bs, D):
    """K goes by rows where a copy has less than 512 bytes: blocks whose runs of 1, 2, 4, 8, 16, 32 and
    64 rows lie on either side for both head sizes, several tiles per sequence, ends inside a tile and
    inside a block."""
    d = _case(8, 2, D, [5, 1, 12, 70, 3], [330, 77, 3, 190, 64 * 3 - 3], bs, seed=300 + bs + D)
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("D,bs", [(64, 4), (64, 6), (128, 2), (128, 4), (128, 12)])
def test_bad_block_ids_in_blocks_of_few_rows(D, bs):
    """Ids out of range among small blocks: their positions are not seen, their neighbours in the same
    tile are."""
    d = _case(8, 2, D, [5, 9], [330, 77], bs, seed=310 + bs + D)
    for b, k in ((0, 0), (0, 17), (0, (330 + 4) // bs), (1, 5)):
        d["table"][b, k] = 10 ** 6 if k % 2 else -1
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == RANGE
    _check(o, d)


@pytest.mark.parametrize("D", [64, 128])
def test_arbitrary_masks_and_rows_that_see_nothing(D):
    d = _case(8, 4, D, [70, 1, 9, 20], [0, 0, 0, 5], 16, seed=50, kind="random")
    d["sees"][0][3] = False
    d["sees"][0][69] = False
    d["sees"][1][0] = False
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)
    got = host_bf16_f64(o)
    assert not got[[3, 69, 70]].any()


def test_bits_above_the_diagonal_are_ignored():
    d = _case(4, 2, 64, [40, 6], [10, 70], 16, seed=51)
    a = _args(d)
    o = fq.attention_tree(*a)
    for s in d["sees"]:
        s |= ~np.tril(np.ones_like(s))
    b = _args(d)
    assert not torch.equal(a[7], b[7])
    assert torch.equal(fq.attention_tree(*b), o)


@pytest.mark.parametrize("Hq,Hkv,n", [(2, 2, 1024), (8, 1, 300), (16, 2, 129)])
def test_no_mask_is_a_chain(Hq, Hkv, n):
    d = _case(Hq, Hkv, 128, [n, 2], [100, 64], 16, seed=52 + n, kind="chain")
    o = fq.attention_tree(*_args(d, mask=False))
    assert fq.check_device_error() == 0
    _check(o, d)
    assert torch.equal(o, fq.attention_tree(*_args(d)))


def test_long_contexts():
    d = _case(8, 2, 128, [33, 4, 1], [20011, 9000, 130], 16, seed=53)
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


def test_many_short_sequences():
    rng = np.random.default_rng(54)
    d = _case(4, 2, 64, rng.integers(0, 4, 700).tolist(), rng.integers(0, 30, 700).tolist(), 8, 54)
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("D,bs", [(64, 7), (64, 16), (128, 7), (128, 32)])
def test_many_items_of_few_tiles(D, bs):
    """Several items per CTA, of one to five position tiles each: what is handed from one item to the
    next (queries, buffers, accumulators) with every parity of the tile counts."""
    rng = np.random.default_rng(68)
    d = _case(32, 16, D, rng.integers(1, 10, 40).tolist(), rng.integers(0, 310, 40).tolist(), bs, 68)
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("sm_scale", [0.0, -0.09, 0.5])
def test_softmax_scales(sm_scale):
    d = _case(8, 2, 128, [12, 40], [200, 333], 16, seed=55)
    o = fq.attention_tree(*_args(d), sm_scale=sm_scale)
    assert fq.check_device_error() == 0
    _check(o, d, sm_scale)


@pytest.mark.parametrize("nodes", [3, 20, 40])
@pytest.mark.parametrize("down", [False, True])
def test_scores_that_grow_along_the_positions(nodes, down):
    """Keys whose size grows (or falls) with the position, queries of one sign: the running maximum
    moves in every tile by up to hundreds of log2 units."""
    d = _case(4, 2, 128, [nodes], [900], 16, seed=56)
    rng = np.random.default_rng(57)
    L = 900 + nodes
    ramp = np.linspace(0.02, 60.0, L)[:, None] * rng.uniform(0.5, 1.5, (L, 2 * 128))
    slots = d["table"][0][np.arange(L) // 16] * 16 + np.arange(L) % 16
    enc = lambda x: (torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn)
                     .view(torch.uint8).numpy())
    d["k"][slots] = enc(ramp[::-1].copy() if down else ramp)
    d["q"][0] = enc(rng.uniform(20, 60, (nodes, 4 * 128)))
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 6), (4, 1, 12), (8, 1, 30)])
def test_nan_codes_that_are_not_seen(Hq, Hkv, n):
    """NaN in every slot no sequence holds and in K and V of nodes that only some rows see: the other
    rows stay exact; a row that sees a NaN value is NaN in that value's dims only, one that sees a NaN
    key is NaN throughout."""
    D = 128
    d = _case(Hq, Hkv, D, [n, 5], [150, 0], 16, seed=58, kind="star")
    d["sees"] = [np.eye(n, dtype=bool), np.eye(5, dtype=bool)]
    slot = lambda b, p: d["table"][b, p // 16] * 16 + p % 16
    held = {slot(0, p) for p in range(150 + n)} | {slot(1, p) for p in range(5)}
    for s in set(range(len(d["k"]))) - held:
        d["k"][s] = d["v"][s] = 0x7F
    clean = dict(d, k=d["k"].copy(), v=d["v"].copy())
    d["v"][slot(0, 150 + 2), 7] = 0xFF                  # node 2: one dim of kv head 0
    d["k"][slot(0, 150 + 4), 3] = 0x7F                  # node 4: key of kv head 0
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    got = host_bf16_f64(o).reshape(n + 5, Hq, D)
    G = Hq // Hkv
    bad = np.zeros((n + 5, Hq, D), bool)
    bad[2, :G, 7] = True
    bad[4, :G] = True
    np.testing.assert_array_equal(np.isnan(got), bad)
    ref = fq.attention_tree(*_args(clean))
    _check(ref, clean)
    same = host_bf16_f64(ref).reshape(n + 5, Hq, D)
    np.testing.assert_array_equal(got[~bad], same[~bad])


def _shared_contexts(B, Hkv, D, ctx, n, seed):
    """B sequences whose contexts lie in the same cache blocks and whose n nodes each lie in blocks of
    their own: long contexts over a small cache."""
    bs, rng = 64, np.random.default_rng(seed)
    assert ctx % bs == 0 and n <= bs
    table = np.concatenate([np.tile(rng.permutation(ctx // bs), (B, 1)),
                            ctx // bs + np.arange(B)[:, None]], axis=1)
    slots = (ctx // bs + B) * bs
    return dict(Hq=Hkv, Hkv=Hkv, D=D, bs=bs, ctx=np.full(B, ctx), nodes=[n] * B, table=table,
                sees=[np.eye(n, dtype=bool)] * B, q=[_codes((n, Hkv * D), rng) for _ in range(B)],
                k=_codes((slots, Hkv * D), rng), v=_codes((slots, Hkv * D), rng),
                s3=np.array([0.011, 0.012, 0.007], np.float32), max_nodes=n, max_len=ctx + n)


def test_nan_values_in_long_contexts():
    """NaN in V of one cached position: exactly that dim of the rows of its kv head is NaN, whatever the
    context's length, and the call takes about as long as without (some 340 position tiles in each
    CTA's share)."""
    B, Hkv, D, ctx, n = 40, 8, 64, 20032, 3
    d = _shared_contexts(B, Hkv, D, ctx, n, 80)
    a = _args(d)
    clean = fq.attention_tree(*a)
    two = dict(d, ctx=d["ctx"][:2], nodes=[n] * 2, table=d["table"][:2], sees=d["sees"][:2], q=d["q"][:2])
    _check(clean[:2 * n], two)
    dirty = list(a)
    dirty[2] = a[2].clone()
    dirty[2][int(d["table"][0, 3]) * 64 + 11, 5 * D + 17] = 0x7F          # position 203, kv head 5
    dirty[2][int(d["table"][0, 311]) * 64 + 63, 2 * D + 40] = 0xFF        # position 19967, kv head 2
    dirty[2][int(d["table"][7, -1]) * 64 + 1, 6 * D] = 0x7F               # node 1 of sequence 7, head 6
    o = fq.attention_tree(*dirty)
    bad = np.zeros((B * n, Hkv, D), bool)
    bad[:, 5, 17] = bad[:, 2, 40] = bad[7 * n + 1, 6, 0] = True
    got, same = (host_bf16_f64(x).reshape(B * n, Hkv, D) for x in (o, clean))
    np.testing.assert_array_equal(np.isnan(got), bad)
    np.testing.assert_array_equal(got[~bad], same[~bad])

    def best(args):
        times = []
        for _ in range(5):
            t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            t[0].record()
            fq.attention_tree(*args)
            t[1].record()
            t[1].synchronize()
            times.append(t[0].elapsed_time(t[1]))
        return min(times)
    slow, fast = best(dirty), best(a)
    assert slow < 3 * fast, f"{slow} ms with NaN, {fast} ms without"
    assert fq.check_device_error() == 0


def test_shares_that_outlast_the_wait_limit():
    """Some 3000 position tiles in each CTA's share of work, a few milliseconds, under waits of 0.25 ms:
    a role that has nothing to do until the next item must not take that for a stall."""
    d = _shared_contexts(40, 8, 64, 64 * 3000, 2, 89)
    a = _args(d)
    o = fq.attention_tree(*a)
    assert fq.check_device_error() == 0
    for _ in range(3):
        got = fq.selftest_attention_tree(64, *a)
        assert fq.check_device_error() == 0
        assert torch.equal(got, o)


@pytest.mark.parametrize("Hq,Hkv,n,D", [(4, 2, 9, 128), (8, 1, 8, 64), (16, 1, 40, 128), (4, 4, 200, 64)])
def test_nan_values_of_context_and_nodes_in_split_items(Hq, Hkv, n, D):
    """One long sequence split over many CTAs: NaN values of cached positions reach every row of their
    kv head, those of a node the rows that see it; repeats of a row and whole row tiles."""
    d = _case(Hq, Hkv, D, [n, 2], [9001, 30], 7, seed=81 + n)
    clean = fq.attention_tree(*_args(d))
    _check(clean, d)
    slot = lambda p: d["table"][0, p // 7] * 7 + p % 7
    G, bad = Hq // Hkv, np.zeros((n + 2, Hq, D), bool)
    for p, g, dim in ((0, 0, 3), (4999, Hkv - 1, D - 1), (9000, 0, 31)):
        d["v"][slot(p), g * D + dim] = 0x7F
        bad[:n, g * G:(g + 1) * G, dim] = True
    for j in {0, n // 2, n - 1}:
        d["v"][slot(9001 + j), (Hkv - 1) * D + 16 + j % 16] = 0xFF
        for i in range(j, n):
            if d["sees"][0][i, j]:
                bad[i, (Hkv - 1) * G:, 16 + j % 16] = True
    got, same = (host_bf16_f64(x).reshape(n + 2, Hq, D) for x in (fq.attention_tree(*_args(d)), clean))
    np.testing.assert_array_equal(np.isnan(got), bad)
    np.testing.assert_array_equal(got[~bad], same[~bad])
    assert fq.check_device_error() == 0


def _rising_case(B, Hq, Hkv, n, D, ctx, shape, seed):
    """_shared_contexts with keys whose level u (a multiple of 2 up to 478, in two dims) follows the
    positions up a ramp, or up and down again, and single large keys in a third dim; query rows that
    take the ramp once, twice, half, negated, not at all, or the large keys.  Three products a score:
    exact in 32 bits."""
    d = _shared_contexts(B, Hkv, D, ctx, n, seed)
    rng = np.random.default_rng(seed + 1)
    G, L = Hq // Hkv, ctx + n
    enc = lambda x: (torch.from_numpy(np.asarray(x, np.float32)).to(torch.float8_e4m3fn)
                     .view(torch.uint8).numpy())
    at = np.linspace(0, 1, L)
    if shape == "tent":
        at = 1 - np.abs(2 * at - 1)
    for g in range(Hkv):
        u = np.clip(np.round((at[:ctx] * 470 + rng.normal(0, 4, ctx)) / 2) * 2, 0, 478).astype(int)
        own = np.clip(np.round((at[ctx:] * 470 + rng.normal(0, 4, (B, n))) / 2) * 2, 0, 478).astype(int)
        big = rng.random(ctx) < 3 / ctx
        big[rng.integers(0, ctx)] = True
        slots = (d["table"][0, :-1][:, None] * 64 + np.arange(64)).reshape(-1)
        d["k"][slots, g * D + 3] = enc(u // 32 * 32)
        d["k"][slots, g * D + 40] = enc(u % 32)
        d["k"][slots, g * D + 63] = enc(np.where(big, 448, 0))
        for b in range(B):
            rows = d["table"][b, -1] * 64 + np.arange(n)
            d["k"][rows, g * D + 3] = enc(own[b] // 32 * 32)
            d["k"][rows, g * D + 40] = enc(own[b] % 32)
            d["k"][rows, g * D + 63] = 0
    d["Hq"] = Hq
    kinds = np.array([[1, 1, 0], [2, 2, 0], [.5, .5, 0], [-1, -1, 0], [0, 0, 0], [1, 1, 1], [1, 1, 0]])
    d["q"] = []
    for b in range(B):
        q = np.zeros((n, Hq, D), np.float32)
        q[:, :, [3, 40, 63]] = kinds[rng.integers(0, len(kinds), (n, Hq))]
        d["q"].append(enc(q).reshape(n, Hq * D))
    d["s3"] = np.array([0.1, 0.1, 0.007], np.float32)
    d["sees"] = [spec.tree_sees([rng.integers(max(-1, i - 5), i) for i in range(n)]) for _ in range(B)]
    return d


def _rescales(d, sm_scale, tiles):
    """How often the accumulators of sequence 0's rows are rescaled over its first `tiles` position tiles
    if a CTA takes them all: the reference moves when a score is more than 8 (in log2 units) above it.
    [rows, repeats] of each kv head, by repeats of the row as the kernel lays them out."""
    val, (D, G) = spec.e4m3_values(), (d["D"], d["Hq"] // d["Hkv"])
    n = d["nodes"][0]
    c2 = sm_scale * float(d["s3"][0]) * float(d["s3"][1]) * np.log2(np.e)
    slots = (d["table"][0][:tiles, None] * 64 + np.arange(64)).reshape(-1)
    rows = min(128, n * G)
    rep = 4 if rows <= 32 else 2 if rows <= 64 else 1
    counts = []
    for h in range(d["Hq"]):
        cols = slice(h // G * D, (h // G + 1) * D)
        z = val[d["q"][0][:, h * D:(h + 1) * D]] @ val[d["k"][slots, cols]].T * c2
        top = z.reshape(n, tiles, rep, 64 // rep).max(axis=3)
        ref, moved = top[:, 0].copy(), np.zeros((n, rep), int)
        for t in range(1, tiles):
            up = top[:, t] > ref + 8
            ref[up] = top[:, t][up]
            moved += up
        counts.append(moved)
    return np.array(counts)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", ["ramp", "tent"])
@pytest.mark.parametrize("Hq,Hkv,n,B", [(8, 4, 3, 30), (16, 4, 10, 30), (8, 2, 30, 60), (8, 2, 50, 30)])
def test_accumulators_rescaled_in_many_tiles(Hq, Hkv, n, B, shape, D):
    """Running maxima that rise by about 10 log2 units a tile (5, 20, or at once by hundreds, in other
    rows), over shares of ten tiles and more: four, two and one repeats of a row, and two row tiles."""
    ctx, sm = 1920, 44.0
    d = _rising_case(B, Hq, Hkv, n, D, ctx, shape, 90 + n)
    moved = _rescales(d, sm, 10)
    assert (moved >= 5).mean() > 0.15 and (moved == 0).mean() > 0.1
    a = _args(d)
    o = fq.attention_tree(*a, sm_scale=sm)
    assert fq.check_device_error() == 0
    two = dict(d, ctx=d["ctx"][:2], nodes=[n] * 2, table=d["table"][:2], sees=d["sees"][:2], q=d["q"][:2])
    _check(o[:2 * n], two, sm)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", ["ramp", "tent"])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 5), (8, 2, 12), (4, 1, 30)])
def test_parts_whose_maxima_lie_far_apart(Hq, Hkv, n, shape, D):
    """One sequence split over many CTAs: their parts' references are tens of log2 units apart."""
    ctx, sm = 6400, 44.0
    d = _rising_case(1, Hq, Hkv, n, D, ctx, shape, 95 + n)
    for scale in (sm, 4.0, 0.3):                        # one part counts, several, all
        o = fq.attention_tree(*_args(d), sm_scale=scale)
        assert fq.check_device_error() == 0
        _check(o, d, scale)


# Small drafts over three or more kv heads.
SHARED = [(3, 3, 20), (4, 4, 64), (10, 5, 16), (32, 8, 16), (32, 8, 7), (12, 4, 21), (40, 5, 8),
          (7, 7, 1), (24, 3, 4)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,most", SHARED)
def test_heads_that_share_a_row_tile(Hq, Hkv, most, D):
    """Drafts from none to as many rows as half a tile holds, contexts from none to several tiles, long
    enough in one sequence that its tiles are split between CTAs."""
    nodes = [1, most, 0, max(1, most // 2), max(1, most - 1), min(3, most), 1]
    d = _case(Hq, Hkv, D, nodes, [0, 1, 40, 63, 64, 3000, 200], 16, seed=70 + Hq + most)
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 4, 9), (4, 4, 40), (6, 3, 30)])
def test_shared_row_tiles_masks_nan_and_growing_scores(Hq, Hkv, n):
    """The same with arbitrary masks and rows that see nothing, with NaN in places that only some rows
    of some heads see, and with scores that grow along the positions."""
    D, G = 128, Hq // Hkv
    d = _case(Hq, Hkv, D, [n, 5], [0, 150], 16, seed=71 + n, kind="random")
    d["sees"][0][n // 2] = False
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)
    assert not host_bf16_f64(o)[n // 2].any()

    d = _case(Hq, Hkv, D, [n, 5], [150, 0], 16, seed=72 + n)
    d["sees"] = [np.eye(n, dtype=bool), np.eye(5, dtype=bool)]
    slot = lambda b, p: d["table"][b, p // 16] * 16 + p % 16
    held = {slot(0, p) for p in range(150 + n)} | {slot(1, p) for p in range(5)}
    for s in set(range(len(d["k"]))) - held:
        d["k"][s] = d["v"][s] = 0x7F
    clean = dict(d, k=d["k"].copy(), v=d["v"].copy())
    d["v"][slot(0, 152), (Hkv - 1) * D + 7] = 0xFF      # node 2: one dim of the last kv head
    d["k"][slot(0, 154), D + 3] = 0x7F                  # node 4: key of kv head 1
    got = host_bf16_f64(fq.attention_tree(*_args(d))).reshape(n + 5, Hq, D)
    bad = np.zeros((n + 5, Hq, D), bool)
    bad[2, (Hkv - 1) * G:, 7] = True
    bad[4, G:2 * G] = True
    np.testing.assert_array_equal(np.isnan(got), bad)
    same = fq.attention_tree(*_args(clean))
    _check(same, clean)
    np.testing.assert_array_equal(got[~bad], host_bf16_f64(same).reshape(n + 5, Hq, D)[~bad])
    assert fq.check_device_error() == 0

    d = _case(Hq, Hkv, D, [n], [900], 16, seed=73 + n)
    rng = np.random.default_rng(74)
    L = 900 + n
    ramp = np.linspace(0.02, 60.0, L)[:, None] * rng.uniform(0.5, 1.5, (L, Hkv * D))
    enc = lambda x: (torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn)
                     .view(torch.uint8).numpy())
    d["k"][d["table"][0][np.arange(L) // 16] * 16 + np.arange(L) % 16] = enc(ramp)
    d["q"][0] = enc(rng.uniform(20, 60, (n, Hq * D)))
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == 0
    _check(o, d)


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (8, 4)])
def test_cache_smaller_than_a_block(Hq, Hkv):
    """No whole block: every id is out of range, nothing is seen, the results are 0."""
    d = _case(Hq, Hkv, 64, [3, 1], [20, 0], 16, seed=75)
    a = _args(d)
    a[1], a[2] = a[1][:9].contiguous(), a[2][:9].contiguous()
    o = fq.attention_tree(*a)
    assert fq.check_device_error() == RANGE
    assert not o.any()


def test_offsets_that_fall_end_the_batch():
    """The sequence whose offsets fall and all behind it have no rows, also where a later one would
    name rows of an earlier one; a sequence with more nodes than max_seq_len has none either."""
    d = _case(8, 2, 128, [4, 5, 6, 3], [100, 90, 80, 10], 16, seed=76)
    for cu, whole in (([0, 4, 2, 3, 6], 1), ([0, 4, 9, 5, 15], 2), ([5, 4, 9, 15, 18], 0)):
        a = _args(d)
        a[6] = i32(cu)
        out = torch.full((18, 8 * 128), 3.0, dtype=torch.bfloat16, device="cuda")
        fq.attention_tree(*a, out=out)
        assert fq.check_device_error() == RANGE
        _check(out, d, seqs=range(whole))
        assert (out[sum(d["nodes"][:whole]):] == 3.0).all()
    a = _args(d)
    a[12] = 5                                           # max_seq_len
    out = torch.full((18, 8 * 128), 3.0, dtype=torch.bfloat16, device="cuda")
    fq.attention_tree(*a, out=out)
    assert fq.check_device_error() == RANGE
    assert (out[9:15] == 3.0).all() and not (out[:9] == 3.0).all(dim=1).any()


def test_bound_on_nodes_above_the_drafts():
    """One graph's bounds over small drafts: the same results to the tolerance as with tight bounds, for
    a bound that takes the single-head form."""
    d = _case(32, 8, 128, [3, 16, 1], [700, 20, 64], 16, seed=77)
    a = _args(d)
    tight = fq.attention_tree(*a)
    d["max_nodes"], d["max_len"] = 200, 1 << 20
    wide = np.full((3, (1 << 20) // 16), -1, np.int32)
    wide[:, :d["table"].shape[1]] = d["table"]
    b = _args(dict(d, table=wide))
    o = fq.attention_tree(*b)
    assert fq.check_device_error() == 0
    _check(o, d)
    _check(tight, d)


def test_strided_and_padded_rows():
    """Leading dimensions wider than the rows, and a capacity beyond the last sequence: what lies
    outside the rows is neither read nor written."""
    d = _case(4, 2, 64, [3, 70, 1], [20, 100, 64], 16, seed=59)
    a = _args(d)
    total, W = sum(d["nodes"]), 4 * 64
    q = torch.full((total + 9, W + 48), 0x7F, dtype=torch.uint8, device="cuda")
    q[:total, :W] = a[0]
    mask = torch.full((total + 9, 5), -1, dtype=torch.int64, device="cuda")
    mask[:total, :a[7].shape[1]] = a[7]
    out = torch.full((total + 9, W + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    a[0], a[7] = q[:, :W], mask
    fq.attention_tree(*a, out=out[:, :W])
    assert fq.check_device_error() == 0
    _check(out[:total, :W].contiguous(), d)
    assert (out[total:] == 3.0).all() and (out[:, W:] == 3.0).all()


def test_cache_beyond_two_gigabytes():
    Hkv, D, bs = 16, 128, 64
    slots = (5 << 30) // (2 * Hkv * D)                  # 2.5 GiB each for K and V
    rng = np.random.default_rng(60)
    blocks = slots // bs
    nodes, ctx = [3, 2], [200, 100]
    table = np.array([[blocks - 1, 0, blocks - 2, blocks // 2], [blocks - 3, blocks - 4, 5, 6]])
    small = _case(16, Hkv, D, nodes, ctx, bs, seed=60)
    k = torch.zeros((slots, Hkv * D), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    for b in range(2):
        for i in range(-(-(ctx[b] + nodes[b]) // bs)):
            at, to = small["table"][b, i] * bs, int(table[b, i]) * bs
            k[to:to + bs] = dev(small["k"][at:at + bs])
            v[to:to + bs] = dev(small["v"][at:at + bs])
    a = _args(small)
    a[1], a[2], a[4] = k, v, i32(table)
    o = fq.attention_tree(*a)
    assert fq.check_device_error() == 0
    _check(o, small)


def test_cache_beyond_two_gigabytes_by_rows():
    """The same where K is copied row by row: blocks of 6 at both ends of 2.5 GiB caches."""
    Hkv, D, bs = 16, 64, 6
    slots = (5 << 30) // (2 * Hkv * D)
    blocks = slots // bs
    nodes, ctx = [3, 2], [200, 100]
    small = _case(16, Hkv, D, nodes, ctx, bs, seed=84)
    table = np.where(small["table"] % 2, small["table"], blocks - 1 - small["table"])
    k = torch.zeros((slots, Hkv * D), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    for b in range(2):
        for i in range(-(-(ctx[b] + nodes[b]) // bs)):
            at, to = small["table"][b, i] * bs, int(table[b, i]) * bs
            k[to:to + bs] = dev(small["k"][at:at + bs])
            v[to:to + bs] = dev(small["v"][at:at + bs])
    a = _args(small)
    a[1], a[2], a[4] = k, v, i32(table)
    o = fq.attention_tree(*a)
    assert fq.check_device_error() == 0
    _check(o, small)


@pytest.mark.parametrize("Hq,Hkv,D,nodes,ctx,bs", [
    (1, 1, 64, 65535, None, 4), (4096, 4096, 64, [2, 1], [5, 70], 3), (128, 1, 128, [7, 0, 20], [300, 3, 65], 16),
    (256, 2, 64, [3, 1], [130, 64], 16), (4, 2, 64, [5, 9], [300, 90], 1 << 14)])
def test_declared_limits(Hq, Hkv, D, nodes, ctx, bs):
    """The largest batch, thousands of kv heads, 128 query heads per kv head, and blocks and length bounds
    far above the lengths."""
    rng = np.random.default_rng(88)
    if ctx is None:
        nodes, ctx = rng.integers(0, 3, nodes).tolist(), rng.integers(0, 20, nodes).tolist()
    d = _case(Hq, Hkv, D, nodes, ctx, bs, seed=88)
    a = _args(d)
    if bs == 1 << 14:
        wide = np.full((2, (1 << 31) // bs), -1, np.int32)
        wide[:, :d["table"].shape[1]] = d["table"]
        a[4], a[12] = i32(wide), 2 ** 31 - 129
    o = fq.attention_tree(*a)
    assert fq.check_device_error() == 0
    _check(o, d)


def test_inputs_out_of_range():
    """A bad block id hides its positions, a context beyond the bound and too many nodes are clamped,
    offsets outside the rows too: recorded, the other sequences as ever."""
    d = _case(8, 2, 128, [4, 5, 6], [100, 90, 80], 16, seed=61)
    d["table"][1, 2] = 10 ** 6
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == RANGE and fq.check_device_error() == 0
    _check(o, d)                                        # the oracle leaves the block out as well
    d["table"][1, 2] = -1
    o = fq.attention_tree(*_args(d))
    assert fq.check_device_error() == RANGE
    _check(o, d)
    d = _case(8, 2, 128, [4, 5, 6], [100, 90, 80], 16, seed=62)
    for where, value in ((5, [100, 10 ** 6, 80]), (5, [100, -5, 80]), (6, [0, 4, 4, 99]),
                         (6, [0, 4, 2, 15])):
        a = _args(d)
        a[where] = i32(value)
        o = fq.attention_tree(*a)
        assert fq.check_device_error() == RANGE
        _check(o, d, seqs=[0])
    a = _args(d)
    a[11] = 4                                           # max_nodes below the other sequences' counts
    out = torch.full((15, 8 * 128), 3.0, dtype=torch.bfloat16, device="cuda")
    fq.attention_tree(*a, out=out)
    assert fq.check_device_error() == RANGE
    _check(out, d, seqs=[0])
    assert (out[8] == 3.0).all() and (out[13:] == 3.0).all()


def test_same_call_same_bits():
    d = _case(32, 8, 128, [16, 3, 9, 11], [3000, 700, 5000, 64], 16, seed=63)
    a = _args(d)
    o = fq.attention_tree(*a)
    ws = torch.full((fq.attention_tree_workspace_bytes(4, 32, 8, 128, 16, d["max_len"]) + 16,), 255,
                    dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(fq.attention_tree(*a, workspace=ws), o)


def test_captured_and_replayed_with_other_lengths():
    """One graph, replayed with the lengths, tables, masks and codes of another batch; a second graph
    over the same workspace in between."""
    d1 = _case(8, 2, 128, [4, 9, 2, 7], [500, 30, 0, 64], 16, seed=64)
    d2 = _case(8, 2, 128, [1, 9, 12, 0], [20, 400, 90, 3], 16, seed=65)
    for d in (d1, d2):                                  # one capacity for both
        d["max_nodes"], d["max_len"] = 12, 600
    a1, a2 = _args(d1), _args(d2)
    width = -(-600 // 16)
    fixed = [torch.zeros((22, 8 * 128), dtype=torch.uint8, device="cuda"),
             torch.zeros((max(len(d1["k"]), len(d2["k"])), 256), dtype=torch.uint8, device="cuda"),
             torch.zeros((max(len(d1["k"]), len(d2["k"])), 256), dtype=torch.uint8, device="cuda"),
             a1[3], i32(np.full((4, width), -1)), i32(np.zeros(4)), i32(np.zeros(5)),
             torch.zeros((22, 1), dtype=torch.int64, device="cuda"), *a1[8:]]
    out = torch.zeros((22, 8 * 128), dtype=torch.bfloat16, device="cuda")
    other = torch.zeros_like(out)
    ws = torch.empty(max(16, fq.attention_tree_workspace_bytes(4, 8, 2, 128, 12, 600)),
                     dtype=torch.uint8, device="cuda")
    fq.attention_tree(*fixed, workspace=ws, out=out)
    graphs = []
    for o in (out, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fq.attention_tree(*fixed, workspace=ws, out=o)
        graphs.append(g)
    for d, a in ((d1, a1), (d2, a2), (d1, a1)):
        for i in (0, 1, 2, 7):
            fixed[i][:a[i].shape[0]] = a[i]
        fixed[4][:, :a[4].shape[1]] = a[4]
        fixed[5].copy_(a[5])
        fixed[6].copy_(a[6])
        for g in graphs:
            g.replay()
        _check(out[:sum(d["nodes"])], d)
        assert torch.equal(out[:sum(d["nodes"])], other[:sum(d["nodes"])])
    assert fq.check_device_error() == 0


def test_on_another_stream():
    d = _case(8, 2, 128, [4, 9], [500, 30], 16, seed=66)
    a = _args(d)
    o = fq.attention_tree(*a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [fq.attention_tree(*a, stream=s) for _ in range(20)]
    torch.cuda.current_stream().wait_stream(s)
    for x in outs:
        assert torch.equal(x, o)


def test_two_calls_at_once():
    """Calls on two streams, each with the workspace it allocates, that run side by side."""
    d1 = _case(8, 2, 128, [4, 9, 30], [500, 30, 2000], 16, seed=86)
    d2 = _case(6, 3, 64, [7, 1], [900, 64], 7, seed=87)
    a1, a2 = _args(d1), _args(d2)
    want = fq.attention_tree(*a1), fq.attention_tree(*a2)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[fq.attention_tree(*a, stream=s) for a, s in zip((a1, a2), streams)] for _ in range(100)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for pair in outs:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])
    assert fq.check_device_error() == 0


def test_speculative_step_end_to_end():
    """Tables, positions, cache write, tree attention, acceptance, and the next step's decode over the
    moved rows, each from the device results of the one before, against the oracle."""
    Hq, Hkv, D, bs, B = 8, 2, 128, 16, 3
    rng = np.random.default_rng(67)
    ctx, nodes = np.array([37, 0, 90]), [6, 3, 8]
    trees = [[-1, 0, 0, 1, 2, 2], [-1, 0, 1], [-1, -1, 0, 1, 2, 3, 4, 4]]
    paths = [[0, 2, 5], [0], [1, 3, 5]]
    table = np.full((B, 8), -1, np.int32)
    table[0, :3], table[2, :6] = [4, 9, 1], [0, 7, 2, 11, 3, 5]
    free = np.array([14, 8, 13, 6, 10, 12], np.int32)
    slots_n, s3 = 16 * bs, np.array([0.02, 0.03, 0.01], np.float32)
    k, v = _codes((slots_n, Hkv * D), rng), _codes((slots_n, Hkv * D), rng)
    dk, dv, dbt, dctx, ds3 = dev(k), dev(v), i32(table), i32(ctx), dev(s3)
    cu, lens, slots, _, left = fq.paged_batch_tables(dctx, i32(nodes), dbt, i32(free), i32([6]), bs,
                                                     20)
    total = sum(nodes)
    mask, pos = fq.tree_mask(i32(np.concatenate(trees + [[0, 0, 0]])), cu, 8, ctx_lens=dctx)
    qkv = torch.from_numpy(rng.standard_normal((20, (Hq + 2 * Hkv) * D), dtype=np.float32)) \
        .to(torch.bfloat16).cuda()
    q = fq.kv_cache_write(qkv, Hq, Hkv, D, slots, ds3, dk, dv)
    o = fq.attention_tree(q, dk, dv, ds3, dbt, dctx, cu, mask, Hq, Hkv, bs, 8, 128)
    path = np.full((B, 4), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    plen = np.array([len(p) for p in paths])
    hk, hv = dk.cpu().numpy().copy(), dv.cpu().numpy().copy()
    new_ctx = fq.kv_cache_accept(dk, dv, dbt, dctx, cu, i32(path), i32(plen), bs)
    assert fq.check_device_error() == 0

    wt, wcu, _, wslots, _, wleft = spec.batch_tables(ctx, nodes, table, bs, free, 6, 20)
    np.testing.assert_array_equal(dbt.cpu().numpy(), wt)
    np.testing.assert_array_equal(slots.cpu().numpy(), wslots)
    assert left.item() == wleft
    bits = qkv.cpu().view(torch.int16).numpy().view(np.uint16)
    wq = oracle.kv_cache_write(bits, Hq, Hkv, D, wslots, s3, k, v)
    np.testing.assert_array_equal(hk, k)
    np.testing.assert_array_equal(hv, v)
    np.testing.assert_array_equal(q.cpu().numpy(), wq)
    sees = [spec.tree_sees(t) for t in trees]
    depth = np.concatenate([s.sum(1) - 1 + c for s, c in zip(sees, ctx)])
    np.testing.assert_array_equal(pos.cpu().numpy()[:total], depth)
    d = dict(Hq=Hq, Hkv=Hkv, D=D, bs=bs, ctx=ctx, nodes=nodes, table=wt, sees=sees, k=k, v=v, s3=s3,
             q=[wq[wcu[b]:wcu[b + 1]] for b in range(B)])
    _check(o[:total], d)
    (wk, wv), wctx = spec.accept([k, v], wt, ctx, path, plen, bs)
    np.testing.assert_array_equal(dk.cpu().numpy(), wk)
    np.testing.assert_array_equal(dv.cpu().numpy(), wv)
    np.testing.assert_array_equal(new_ctx.cpu().numpy(), wctx)
    # the accepted path is now an ordinary context: one decode step sees the same rows as the path's
    # last node did, in the order of the path
    last = torch.stack([q[wcu[b] + paths[b][-1]] for b in range(B)])
    step = fq.attention_decode(last, dk, dv, ds3, dbt, new_ctx, Hq, Hkv, bs, 128)
    one = dict(d, ctx=wctx - 1, nodes=[1] * B, sees=[np.ones((1, 1), bool)] * B, k=wk, v=wv,
               q=[last[b:b + 1].cpu().numpy() for b in range(B)])
    _check(step, one)
    np.testing.assert_allclose(host_bf16_f64(step),
                               host_bf16_f64(o)[[wcu[b] + paths[b][-1] for b in range(B)]],
                               rtol=2.0 ** -6, atol=2.0 ** -8)


def test_speculative_loop_in_a_graph():
    """Steps of a whole loop, captured once and replayed: tables over the blocks held, masks, cache write,
    attention, acceptance, and the lengths, stack height and held blocks handed on by the graph itself.
    Every result of every step against the oracle; no block is lost although most nodes are rejected."""
    Hq, Hkv, D, bs, B, most, cap, width = 8, 2, 64, 4, 3, 8, 24, 24
    rng = np.random.default_rng(85)
    ctx, s3 = np.array([13, 0, 30]), np.array([0.02, 0.03, 0.01], np.float32)
    table, ids = np.full((B, width), -1, np.int32), rng.permutation(30).astype(np.int32)
    have, at = -(-ctx // bs), 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = np.concatenate([ids[at:], np.zeros(at, np.int32)])
    k, v = _codes((30 * bs, Hkv * D), rng), _codes((30 * bs, Hkv * D), rng)
    dk, dv, dbt, dctx, ds3, dfree = dev(k), dev(v), i32(table), i32(ctx), dev(s3), i32(free)
    count, held = i32([30 - at]), i32(np.zeros(B))
    new, parents = i32(np.zeros(B)), i32(np.full(cap, -1))
    path, plen = i32(np.zeros((B, most))), i32(np.zeros(B))
    qkv = torch.zeros((cap, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")

    def step():
        cu, lens, slots, _, left, now = fq.paged_batch_tables(dctx, new, dbt, dfree, count, bs, cap,
                                                              held_blocks=held)
        mask, pos = fq.tree_mask(parents, cu, most, ctx_lens=dctx)
        q = fq.kv_cache_write(qkv, Hq, Hkv, D, slots, ds3, dk, dv)
        o = fq.attention_tree(q, dk, dv, ds3, dbt, dctx, cu, mask, Hq, Hkv, bs, most, width * bs)
        lens = fq.kv_cache_accept(dk, dv, dbt, dctx, cu, path, plen, bs)
        for old, x in ((count, left), (held, now), (dctx, lens)):
            old.copy_(x)
        return slots, pos, q, o
    step()                                               # no nodes: everything stays as it is
    assert held.cpu().numpy().tolist() == have.tolist() and dctx.cpu().numpy().tolist() == ctx.tolist()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slots, pos, q, o = step()
    wfree, wcount, wheld, wtable = free, 30 - at, have, table
    for _ in range(12):
        nodes = rng.integers(0, most + 1, B)
        trees = [[int(rng.integers(max(-1, i - 4), i)) for i in range(n)] for n in nodes]
        paths = []
        for t in trees:                                  # from the root to some node, cut short
            p, i = [], len(t) - 1
            while i >= 0:
                p.append(i)
                i = t[i]
            paths.append(p[::-1][:rng.integers(0, 3)])
        total = int(nodes.sum())
        new.copy_(i32(nodes))
        parents[:total] = i32(np.concatenate([np.array(t, int) for t in trees]))
        for b, p in enumerate(paths):
            path[b, :len(p)] = i32(p)
        plen.copy_(i32([len(p) for p in paths]))
        qkv.copy_(torch.from_numpy(rng.standard_normal(tuple(qkv.shape), dtype=np.float32)))
        g.replay()
        assert fq.check_device_error() == 0
        wtable, wcu, _, wslots, _, wcount, wheld = spec.batch_tables(ctx, nodes, wtable, bs, wfree, wcount,
                                                                     cap, held=wheld)
        np.testing.assert_array_equal(slots.cpu().numpy(), wslots)
        np.testing.assert_array_equal(dbt.cpu().numpy(), wtable)
        bits = qkv.cpu().view(torch.int16).numpy().view(np.uint16)
        wq = oracle.kv_cache_write(bits, Hq, Hkv, D, wslots, s3, k, v)
        np.testing.assert_array_equal(q.cpu().numpy()[:total], wq[:total])
        sees = [spec.tree_sees(t) for t in trees]
        np.testing.assert_array_equal(
            pos.cpu().numpy()[:total], np.concatenate([s.sum(1) - 1 + c for s, c in zip(sees, ctx)]))
        d = dict(Hq=Hq, Hkv=Hkv, D=D, bs=bs, ctx=ctx, nodes=nodes, table=wtable, sees=sees, k=k, v=v,
                 s3=s3, q=[wq[wcu[b]:wcu[b + 1]] for b in range(B)])
        _check(o[:total], d)
        (k, v), ctx = spec.accept([k, v], wtable, ctx, paths, [len(p) for p in paths], bs)
        for got, ref in ((dk, k), (dv, v), (dctx, ctx), (held, wheld), (count, [wcount])):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
        kept = np.concatenate([wtable[b, :wheld[b]] for b in range(B)] + [wfree[:wcount]])
        np.testing.assert_array_equal(np.sort(kept), np.arange(30))
