"""GPU parity of the integer operators of a speculative-decoding step (block tables and slot maps,
ancestor masks, the move of accepted rows) against the oracle, equal to the last bit: batches from one
request to more than a CTA's threads, block sizes 1, 5, 16 and 64, empty requests and trees, padded
capacities, chains of 1024 nodes, overlapping moves, and inputs that break a rule (recorded, clamped,
nothing outside the buffers)."""
import numpy as np
import pytest
import torch

import fp8_blockwise_w8a8_b200 as fq
from oracle import speculative as spec

pytestmark = pytest.mark.gpu
RANGE = 9


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def host(t):
    return t.cpu().numpy()


# --- block tables and slot maps ------------------------------------------------------------------

def _tables_case(B, bs, ctx_hi, new_hi, seed, spare=7):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_hi + 1, B), rng.integers(0, new_hi + 1, B)
    have, want = -(-ctx // bs), -(-(ctx + new) // bs)
    perm = rng.permutation(int(want.sum()) + spare).astype(np.int32)
    table = np.full((B, max(1, int(want.max(initial=0))) + 1), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    return ctx, new, table, perm[at:]


def _check_tables(ctx, new, table, bs, free, count, max_tokens):
    want = spec.batch_tables(ctx, new, table, bs, free, count, max_tokens)
    bt = i32(table)
    cu, lens, slots, pos, left = fq.paged_batch_tables(i32(ctx), i32(new), bt, i32(free),
                                                       i32([count]), bs, max_tokens)
    for got, ref in zip((bt, cu, lens, slots, pos, left), want):
        np.testing.assert_array_equal(host(got), ref)


@pytest.mark.parametrize("B,bs,ctx_hi,new_hi", [
    (1, 16, 0, 1), (1, 5, 40, 3000), (7, 1, 9, 4), (64, 16, 4096, 1), (513, 16, 100, 9),
    (1500, 64, 500, 40), (3, 16, 20, 20000)])
def test_tables(B, bs, ctx_hi, new_hi):
    ctx, new, table, free = _tables_case(B, bs, ctx_hi, new_hi, B + bs)
    total = int(new.sum())
    _check_tables(ctx, new, table, bs, free, len(free), total + 77)
    _check_tables(ctx, new, table, bs, free, len(free) - 3, total)
    assert fq.check_device_error() == 0


def test_tables_largest_batch():
    ctx, new, table, free = _tables_case(16384, 16, 30, 3, 1)
    _check_tables(ctx, new, table, 16, free, len(free), int(new.sum()) + 1)
    assert fq.check_device_error() == 0


def test_tables_no_requests_and_no_tokens():
    e = np.zeros(0, np.int32)
    cu, lens, slots, pos, left = fq.paged_batch_tables(i32(e), i32(e), i32(np.zeros((0, 3))),
                                                       i32([4, 2]), i32([2]), 16, 5)
    assert host(cu).tolist() == [0] and host(left).tolist() == [2]
    assert host(slots).tolist() == [-1] * 5 and host(pos).tolist() == [0] * 5
    cu, lens, slots, pos, left = fq.paged_batch_tables(i32([5, 0]), i32([0, 0]),
                                                       i32([[1], [-1]]), i32(e), i32([0]), 16, 0)
    assert host(cu).tolist() == [0, 0, 0] and host(lens).tolist() == [5, 0]
    assert slots.numel() == 0 and host(left).tolist() == [0]
    assert fq.check_device_error() == 0


def test_tables_free_stack_too_short():
    ctx, new, table, free = _tables_case(40, 16, 100, 50, 5)
    total = int(new.sum())
    _check_tables(ctx, new, table, 16, free, 20, total)
    assert fq.check_device_error() == RANGE
    _check_tables(ctx, new, table, 16, free, 0, total)
    assert fq.check_device_error() == RANGE and fq.check_device_error() == 0


def test_tables_lengths_out_of_range():
    """A negative length counts as 0, one beyond the table is cut at its end, tokens beyond max_tokens
    are cut off, and a stack height outside the stack is clamped; all recorded."""
    table = np.array([[3, -1], [5, -1], [0, -1], [6, -1]], np.int32)
    args = lambda ctx, new, count, cap: (i32(ctx), i32(new), i32(table), i32([9, 8, 7]),
                                         i32([count]), 4, cap)
    out = fq.paged_batch_tables(*args([-2, 3, 2, 4], [2, -1, 99, 0], 3, 9))
    assert fq.check_device_error() == RANGE
    assert host(out[0]).tolist() == [0, 2, 2, 8, 8] and host(out[1]).tolist() == [2, 3, 8, 4]
    # request 0 starts at 0: its first block is new (7); request 2 goes on in block 0, then 8
    assert host(out[2]).tolist() == [28, 29, 2, 3, 32, 33, 34, 35, -1]
    assert host(out[3]).tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 0] and host(out[4]).tolist() == [1]
    out = fq.paged_batch_tables(*args([1, 3, 1, 1], [2, 2, 2, 2], 3, 5))       # 8 tokens into 5
    assert fq.check_device_error() == RANGE
    assert host(out[0]).tolist() == [0, 2, 4, 5, 5] and host(out[1]).tolist() == [3, 5, 2, 1]
    assert host(out[2]).tolist() == [13, 14, 23, 28, 1] and host(out[4]).tolist() == [2]
    out = fq.paged_batch_tables(*args([4, 4, 4, 4], [1, 0, 0, 0], 4, 1))       # 4 of 3 entries
    assert fq.check_device_error() == RANGE
    assert host(out[2]).tolist() == [28] and host(out[4]).tolist() == [2]


def test_tables_step_after_step_in_a_graph():
    """A captured decode step, replayed: the results become the next step's inputs on the device."""
    B, bs, cap = 5, 4, 12
    rng = np.random.default_rng(8)
    ctx, new = i32([0, 3, 4, 11, 6]), i32([1, 2, 0, 3, 1])
    table = np.full((B, 16), -1, np.int32)
    free = rng.permutation(80).astype(np.int32)
    for b, c in enumerate(host(ctx)):
        table[b, :-(-c // bs)] = 100 + 10 * b + np.arange(-(-c // bs))
    bt, fb, count = i32(table), i32(free), i32([80])
    out = fq.paged_batch_tables(ctx, new, bt.clone(), fb, count, bs, cap)      # buffers
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        fq.paged_batch_tables(ctx, new, bt, fb, count, bs, cap, out=out)
        ctx.copy_(out[1])
        count.copy_(out[4])
    c, t, k = host(ctx).copy(), table, 80
    for step in range(6):
        n = rng.integers(0, 3, B)
        new.copy_(i32(n))
        g.replay()
        t, cu, lens, slots, pos, k = spec.batch_tables(c, n, t, bs, free, k, cap)
        for got, ref in zip((bt, *out), (t, cu, lens, slots, pos, k)):
            np.testing.assert_array_equal(host(got), ref)
        c = lens
    assert fq.check_device_error() == 0


@pytest.mark.parametrize("bs,spare", [(16, 40), (5, 50), (1, 330)])
def test_many_steps_with_rejections_keep_every_block(bs, spare):
    """Speculative steps of tables and acceptance, each from the device results of the one before, with
    most nodes rejected: after every step each block id is in exactly one held place or on the stack,
    the requests hold no more than their longest reach so far, and requests that end give back what
    they hold.  More steps than the stack could feed if the blocks of rejected nodes were popped anew."""
    B, n_hi, steps, width = 9, 16, 60, 400
    rng = np.random.default_rng(bs)
    ctx = rng.integers(0, 40, B)
    have = -(-ctx // bs)
    perm = rng.permutation(int(have.sum()) + B * (-(-n_hi // bs) + 1) + spare).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    stack = np.zeros(len(perm), np.int32)
    stack[:len(perm) - at] = perm[at:]
    dctx, dbt, dfree = i32(ctx), i32(table), i32(stack)
    count, held = i32([len(perm) - at]), i32(np.zeros(B))
    cache = torch.zeros((len(perm) * bs, 16), dtype=torch.uint8, device="cuda")
    reach, popped_anew = have.copy(), 0
    for step in range(steps):
        n = rng.integers(0, n_hi + 1, B)
        accepted = np.minimum(n, rng.integers(0, 2, B))          # at most one
        wtable, wcu, wlens, wslots, _, wleft, wheld = spec.batch_tables(
            ctx, n, host(dbt), bs, host(dfree), int(host(count)[0]), B * n_hi, held=host(held))
        cu, lens, slots, _, count, held = fq.paged_batch_tables(dctx, i32(n), dbt, dfree, count, bs,
                                                                B * n_hi, held_blocks=held)
        for got, ref in zip((dbt, cu, lens, slots, count, held),
                            (wtable, wcu, wlens, wslots, [wleft], wheld)):
            np.testing.assert_array_equal(host(got), ref)
        assert (host(slots)[:n.sum()] >= 0).all()
        path = np.array([[max(0, k - 1)] for k in n])            # the last node, where there is one
        dctx = fq.kv_cache_accept(cache, cache.clone(), dbt, dctx, cu, i32(path), i32(accepted), bs)
        popped_anew += (-(-(ctx + n) // bs) - -(-ctx // bs)).sum()
        reach = np.maximum(reach, -(-(ctx + n) // bs))
        np.testing.assert_array_equal(host(held), reach)
        ctx = ctx + accepted
        np.testing.assert_array_equal(host(dctx), ctx)
        ids = np.concatenate([host(dbt)[b, :h] for b, h in enumerate(host(held))] +
                             [host(dfree)[:host(count)[0]]])
        np.testing.assert_array_equal(np.sort(ids), np.arange(len(perm)))
        if step % 20 == 19:                                      # request 4 ends, another begins
            h, c = int(host(held)[4]), int(host(count)[0])
            dfree[c:c + h] = dbt[4, :h]
            count += h
            held[4], dctx[4], ctx[4], reach[4] = 0, 0, 0, 0
    assert popped_anew > len(perm) - have.sum()
    assert fq.check_device_error() == 0


def test_tables_held_blocks_where_the_stack_runs_short():
    """What the stack cannot give is not held, and is popped by the next call; counts out of range are
    clamped and recorded; a context beyond the count holds its own blocks."""
    table = [[3, 5, -1], [6, 7, 9], [0, -1, -1]]
    bt = i32(table)
    args = lambda ctx, new, free, count: (i32(ctx), i32(new), bt, i32(free), i32([count]), 4, 16)
    out = fq.paged_batch_tables(*args([4, 1, 4], [6, 2, 8], [8, 2], 2), held_blocks=i32([2, 3, 0]))
    assert fq.check_device_error() == RANGE
    want = spec.batch_tables([4, 1, 4], [6, 2, 8], table, 4, [8, 2], 2, 16, held=[2, 3, 0])
    for got, ref in zip((bt, *out), (*want[:5], [want[5]], want[6])):
        np.testing.assert_array_equal(host(got), ref)
    out = fq.paged_batch_tables(*args([4, 1, 4], [6, 2, 8], [1], 1), held_blocks=out[5])
    assert fq.check_device_error() == 0
    assert host(bt).tolist() == [[3, 5, 2], [6, 7, 9], [0, 8, 1]]
    assert host(out[5]).tolist() == [3, 3, 3] and host(out[4]).tolist() == [0]
    out = fq.paged_batch_tables(*args([4, 1, 4], [6, 2, 8], [1], 1), held_blocks=i32([-1, 3, 99]))
    assert fq.check_device_error() == RANGE
    assert host(out[5]).tolist() == [2, 3, 3] and host(out[4]).tolist() == [0]
    assert host(bt).tolist() == [[3, 1, -1], [6, 7, 9], [0, 8, 1]]
    assert host(out[2])[:6].tolist() == [4, 5, 6, 7, -1, -1]


def test_tables_held_blocks_of_a_large_batch():
    """More requests than a CTA has threads and more tokens than one thread's groups, with counts at
    random between the context's blocks and the table's end."""
    ctx, new, table, free = _tables_case(1500, 64, 500, 300, 21)
    rng = np.random.default_rng(22)
    have, want = -(-ctx // 64), -(-(ctx + new) // 64)
    held = rng.integers(0, want + 2)
    for b in range(1500):                                        # ids for the blocks held beyond
        for k in range(have[b], held[b]):
            table[b, k] = 10 ** 6 + 100 * b + k
    total = int(new.sum()) + 5
    assert total > 2 * 148 * 512
    ref = spec.batch_tables(ctx, new, table, 64, free, len(free), total, held=held)
    bt, out = i32(table), (i32(np.zeros(1501)), i32(np.zeros(1500)), torch.empty(
        total, dtype=torch.int64, device="cuda"), torch.empty(total, dtype=torch.int64, device="cuda"),
        i32([0]), i32(np.zeros(1500)))
    got = fq.paged_batch_tables(i32(ctx), i32(new), bt, i32(free), i32([len(free)]), 64, total, out=out,
                                held_blocks=i32(held))
    for x, y in zip((bt, *got), (*ref[:5], [ref[5]], ref[6])):
        np.testing.assert_array_equal(host(x), y)
    assert got[5].data_ptr() == out[5].data_ptr() and fq.check_device_error() == 0


# --- ancestor masks -------------------------------------------------------------------------------

def _parents(n, rng, kind):
    if kind == "chain":
        return np.arange(-1, n - 1)
    if kind == "star":
        return np.full(n, -1)
    return np.array([rng.integers(max(-1, i - 9), i) for i in range(n)], np.int64)


def _check_mask(sizes, max_nodes, kind, seed, pad=0):
    rng = np.random.default_rng(seed)
    trees = [_parents(n, rng, kind) for n in sizes]
    words = -(-max_nodes // 64)
    cu = np.concatenate([[0], np.cumsum(sizes)])
    total = int(cu[-1]) + pad
    parents = np.concatenate(trees + [np.full(pad, 10 ** 6)])
    ctx = rng.integers(0, 10 ** 6, len(sizes))
    mask = torch.full((total, words + 1), -7, dtype=torch.int64, device="cuda")
    pos = torch.full((total,), -7, dtype=torch.int64, device="cuda")
    fq.tree_mask(i32(parents), i32(cu), max_nodes, ctx_lens=i32(ctx), out_mask=mask[:, :words],
                 out_positions=pos)
    want, wpos = np.full((total, words + 1), -7), np.full(total, -7)
    for b, t in enumerate(trees):
        sees = spec.tree_sees(t)
        want[cu[b]:cu[b + 1], :words] = spec.pack_bits(sees, words)
        wpos[cu[b]:cu[b + 1]] = ctx[b] + sees.sum(1) - 1
    np.testing.assert_array_equal(host(mask), want)
    np.testing.assert_array_equal(host(pos), wpos)
    assert fq.check_device_error() == 0


@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("sizes,max_nodes", [
    ([1], 1), ([0, 1, 2, 0, 16, 7], 16), ([63, 64, 65, 1], 65), ([256, 3, 0, 200], 256),
    ([257, 511], 512), ([1024, 1, 1000], 1024)])
def test_mask(sizes, max_nodes, kind):
    _check_mask(sizes, max_nodes, kind, 3, pad=5)


def test_mask_many_sequences():
    rng = np.random.default_rng(4)
    _check_mask(rng.integers(0, 12, 3000).tolist(), 40, "random", 5)


def test_mask_without_contexts_and_nodes():
    mask, pos = fq.tree_mask(i32([-1, 0, 0]), i32([0, 3]), 8)
    assert host(mask)[:, 0].tolist() == [1, 3, 5] and host(pos).tolist() == [0, 1, 1]
    mask, pos = fq.tree_mask(i32(np.zeros(0)), i32([0, 0]), 8)
    assert mask.shape == (0, 1) and pos.shape == (0,)
    assert fq.check_device_error() == 0


def test_mask_bad_parents_and_offsets():
    """A parent that is not before its child counts as the context; a sequence above max_nodes is
    written up to there; offsets outside the rows are clamped."""
    mask, _ = fq.tree_mask(i32([-1, 1, -2, 2]), i32([0, 4]), 4)
    assert fq.check_device_error() == RANGE
    assert host(mask)[:, 0].tolist() == [1, 2, 4, 12]
    out = torch.full((6, 1), -7, dtype=torch.int64, device="cuda")
    fq.tree_mask(i32([-1, 0, 1, 2, -1, 0]), i32([0, 4, 99]), 3, out_mask=out)
    assert fq.check_device_error() == RANGE
    assert host(out)[:, 0].tolist() == [1, 3, 7, -7, 1, 3]
    out.fill_(-7)
    fq.tree_mask(i32([-1, 0, 1, 2, -1, 0]), i32([-3, 2, 1]), 3, out_mask=out)
    assert fq.check_device_error() == RANGE
    assert host(out)[:, 0].tolist() == [1, 3, -7, -7, -7, -7]


def test_mask_offsets_that_fall_end_the_batch():
    """Later sequences would name rows of an earlier one: nothing of theirs is written."""
    par = [-1, 0, 1, 2, -1, 0, 0, -1, 0]
    for cu, rows in (([0, 4, 2, 3, 6], 4), ([0, 3, 5, 4, 9], 5), ([4, 2, 9, 9, 9], 0)):
        out = torch.full((9, 1), -7, dtype=torch.int64, device="cuda")
        pos = torch.full((9,), -7, dtype=torch.int64, device="cuda")
        fq.tree_mask(i32(par), i32(cu), 8, out_mask=out, out_positions=pos)
        assert fq.check_device_error() == RANGE
        assert (host(out)[rows:] == -7).all() and (host(pos)[rows:] == -7).all()
        assert (host(out)[:rows] != -7).all()


def test_mask_depths_of_long_trees():
    """Positions of trees whose nodes' chains cross several words of the mask."""
    rng = np.random.default_rng(9)
    par = np.concatenate([np.arange(-1, 699), [rng.integers(max(0, i - 3), i) for i in range(700, 1024)]])
    mask, pos = fq.tree_mask(i32(par), i32([0, 1024]), 1024, ctx_lens=i32([50]))
    sees = spec.tree_sees(par)
    np.testing.assert_array_equal(host(mask), spec.pack_bits(sees, 16))
    np.testing.assert_array_equal(host(pos), 50 + sees.sum(1) - 1)
    assert fq.check_device_error() == 0


@pytest.mark.parametrize("cap", [151552, 151553, 400001])
def test_tables_many_tokens(cap):
    """Around and above the size from which a thread takes four tokens, with capacities that leave a
    partial group at the end, an unaligned slot array among them."""
    rng = np.random.default_rng(cap)
    B, bs = 37, 24
    new = rng.multinomial(cap - 5, rng.dirichlet(np.ones(B)))
    ctx = rng.integers(0, 900, B)
    ctx[3], new[7] = 0, 0
    total = int(new.sum())
    have, want = -(-ctx // bs), -(-(ctx + new) // bs)
    perm = rng.permutation(int(want.sum())).astype(np.int32)
    table = np.full((B, int(want.max())), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    free = perm[at:]
    ref = spec.batch_tables(ctx, new, table, bs, free, len(free), cap)
    for skew in (0, 1):
        slots = torch.empty(cap + skew, dtype=torch.int64, device="cuda")[skew:]
        pos = torch.empty(cap, dtype=torch.int64, device="cuda")
        bt = i32(table)
        out = (i32(np.zeros(B + 1)), i32(np.zeros(B)), slots, pos, i32([0]))
        fq.paged_batch_tables(i32(ctx), i32(new), bt, i32(free), i32([len(free)]), bs, cap, out=out)
        for got, want_ in zip((bt, *out), ref):
            np.testing.assert_array_equal(host(got), want_)
    assert total <= cap and fq.check_device_error() == 0


# --- accepted rows --------------------------------------------------------------------------------

def _accept_case(B, bs, row, layers, seed, n_hi=20, path_hi=12):
    rng = np.random.default_rng(seed)
    n, ctx = rng.integers(0, n_hi + 1, B), rng.integers(0, 50, B)
    width = max(1, int((-(-(ctx + n) // bs)).max()))
    table = rng.permutation(B * width + 3)[:B * width].reshape(B, width).astype(np.int32)
    slots = (B * width + 3) * bs
    k, v = (rng.integers(0, 256, (layers, slots, row)).astype(np.uint8) for _ in range(2))
    path, plen = np.full((B, path_hi), -9, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        plen[b] = rng.integers(0, min(path_hi, n[b]) + 1)
        path[b, :plen[b]] = np.sort(rng.permutation(n[b])[:plen[b]])
    return k, v, table, ctx, n, path, plen


@pytest.mark.parametrize("B,bs,row,layers", [
    (1, 16, 16, 1), (9, 1, 48, 2), (30, 7, 1024, 1), (12, 64, 272, 5), (3, 16, 4096, 2)])
def test_accept(B, bs, row, layers):
    k, v, table, ctx, n, path, plen = _accept_case(B, bs, row, layers, B)
    (wk, wv), lens = spec.accept([k, v], table, ctx, path, plen, bs)
    dk, dv = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    cu = i32(np.concatenate([[0], np.cumsum(n)]))
    if layers == 1:
        dk, dv = dk[0], dv[0]
        wk, wv = wk[0], wv[0]
    got = fq.kv_cache_accept(dk, dv, i32(table), i32(ctx), cu, i32(path), i32(plen), bs)
    np.testing.assert_array_equal(host(got), lens)
    np.testing.assert_array_equal(host(dk), wk)
    np.testing.assert_array_equal(host(dv), wv)
    assert fq.check_device_error() == 0


def test_accept_long_overlapping_path():
    """1000 of 1024 nodes, in place from some index on, shifted by ever more behind it."""
    rng = np.random.default_rng(6)
    path = np.sort(rng.permutation(1024)[:1000])
    path[:30] = np.arange(30)
    k = rng.integers(0, 256, (1, 1100, 32)).astype(np.uint8)
    table = rng.permutation(110).reshape(1, 110).astype(np.int32)
    (wk, wv), lens = spec.accept([k, k], table, [13], [path], [1000], 10)
    dk, dv = torch.from_numpy(k).cuda(), torch.from_numpy(k).cuda()
    fq.kv_cache_accept(dk, dv, i32(table), i32([13]), i32([0, 1024]), i32(path[None]), i32([1000]), 10)
    np.testing.assert_array_equal(host(dk), wk)
    np.testing.assert_array_equal(host(dv), wv)
    assert fq.check_device_error() == 0


def test_accept_bad_paths_move_nothing():
    """Paths that repeat or fall, leave the nodes or are too long, a bad block and a bad context: those
    sequences keep their rows and lengths, the good one beside them moves."""
    B, bs = 7, 4
    rng = np.random.default_rng(7)
    table = np.arange(B * 4).reshape(B, 4).astype(np.int32)
    k = rng.integers(0, 256, (B * 16, 16)).astype(np.uint8)
    path = np.array([[0, 2, 2], [2, 1, 3], [0, 1, 5], [0, 2, 4], [0, 2, 4], [0, 2, 4], [0, 2, 4]])
    plen, ctx = [3, 3, 3, 4, 3, 3, 3], [1, 2, 3, 4, 5, 14, 7]
    table[4, 2] = 10 ** 6                               # holds the accepted node 4 of sequence 4
    (wk, _), _ = spec.accept([k, k], table[6:], [7], path[6:], [3], bs)
    dk, dv = torch.from_numpy(k).cuda(), torch.from_numpy(k).cuda()
    got = fq.kv_cache_accept(dk, dv, i32(table), i32(ctx), i32(np.arange(B + 1) * 5), i32(path),
                             i32(plen), bs)
    assert fq.check_device_error() == RANGE
    assert host(got).tolist() == [1, 2, 3, 4, 5, 14, 10]
    np.testing.assert_array_equal(host(dk), wk)
    np.testing.assert_array_equal(host(dv), wk)
