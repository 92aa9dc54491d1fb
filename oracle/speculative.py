"""Oracle of the speculative-decoding operators (test infrastructure only): numpy, 64 bits, written
from the definitions in include/fp8q.h, one sequence, node and position at a time where speed
allows."""
import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of every E4M3 code (bias 7, no infinities, 0x7F and 0xFF NaN), from the format."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        mag = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 127 == 127 else (-mag if c & 128 else mag)
    return v


def batch_tables(ctx, new, table, block_size, free_blocks, free_count, max_tokens, held=None):
    """(table, cu, seq_lens, slots, positions, free_left) for lengths within the table and tokens
    within max_tokens; blocks that the stack cannot give are -1.  `held`: the blocks that each request
    holds already; their number afterwards is appended to the results."""
    table = np.array(table, np.int64)
    stack = list(free_blocks[:free_count])
    slots, positions, cu, after = [], [], [0], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        have = max(-(-c // block_size), 0 if held is None else held[b])
        for k in range(have, -(-(c + n) // block_size)):
            have += bool(stack)
            table[b, k] = stack.pop() if stack else -1
        after.append(have)
        for p in range(c, c + n):
            blk = table[b, p // block_size]
            slots.append(-1 if blk < 0 else blk * block_size + p % block_size)
            positions.append(p)
        cu.append(cu[-1] + n)
    behind = max_tokens - len(slots)
    return (table, np.array(cu), np.array(ctx, np.int64) + np.array(new, np.int64),
            np.array(slots + [-1] * behind, np.int64),
            np.array(positions + [0] * behind, np.int64), len(stack),
            *([] if held is None else [np.array(after, np.int64)]))


def tree_sees(parents) -> np.ndarray:
    """bool [n, n]: node i sees j (itself and its ancestors)."""
    n = len(parents)
    sees = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = parents[j]
    return sees


def pack_bits(sees, words) -> np.ndarray:
    """bool [n, m] -> int64 [n, words], bit j of a row in word j // 64."""
    n, m = sees.shape
    out = np.zeros((n, words), np.uint64)
    for j in range(m):
        out[:, j // 64] |= sees[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)


def attention(q, k_cache, v_cache, scale3, table, ctx, sees, Hq, Hkv, block_size, sm_scale=None):
    """Tree attention in float64.  q: list of code arrays [n_b, Hq * D]; sees: list of bool [n_b, n_b]
    (taken below the diagonal).  Returns lists of out, absref (both [n_b, Hq * D]) and zabs, L
    ([n_b, Hq] and [n_b]): the largest |scale| sum_d |q k| and the number of positions seen."""
    val = e4m3_values()
    G, D = Hq // Hkv, k_cache.shape[1] // Hkv
    sq, sk, sv = (float(x) for x in scale3)
    sm = float(np.float32(1.0 / np.sqrt(D) if sm_scale is None else sm_scale))  # an fp32 argument
    outs, absrefs, zabss, counts = [], [], [], []
    for b, codes in enumerate(q):
        n, c = len(codes), ctx[b]
        pos = np.arange(c + n)
        blk = np.asarray(table[b], np.int64)[pos // block_size]
        nblocks = len(k_cache) // block_size
        there = (blk >= 0) & (blk < nblocks)
        slot = np.where(there, blk, 0) * block_size + pos % block_size
        see = np.concatenate([np.ones((n, c), bool), np.tril(sees[b])], axis=1) & there
        out, absref = np.zeros((n, Hq * D)), np.zeros((n, Hq * D))
        zabs = np.zeros((n, Hq))
        for h in range(Hq):
            g, cols = h // G, slice(h * D, (h + 1) * D)
            k = val[k_cache[slot, g * D:(g + 1) * D]]
            v = val[v_cache[slot, g * D:(g + 1) * D]] * sv
            qh = val[codes[:, cols]]
            for i in range(n):
                s = see[i]
                if not s.any():
                    continue
                z = k[s] @ qh[i] * (sm * sq * sk)
                p = np.exp(z - z.max())
                p /= p.sum()
                out[i, cols] = p @ v[s]
                absref[i, cols] = p @ np.abs(v[s])
                zabs[i, h] = abs(sm * sq * sk) * (np.abs(k[s]) @ np.abs(qh[i])).max()
        outs.append(out)
        absrefs.append(absref)
        zabss.append(zabs)
        counts.append(see.sum(axis=1))
    return outs, absrefs, zabss, counts


def accept(caches, table, ctx, path, path_lens, block_size):
    """The caches [..., slots, row] after the moves, one after the other, and the new lengths."""
    caches = [c.copy() for c in caches]
    for b, c in enumerate(ctx):
        for k in range(path_lens[b]):
            f, t = c + path[b][k], c + k
            src = table[b][f // block_size] * block_size + f % block_size
            dst = table[b][t // block_size] * block_size + t % block_size
            for cache in caches:
                cache[..., dst, :] = cache[..., src, :]
    return caches, np.array(ctx) + np.array(path_lens)
