"""Speculative decoding over the paged FP8 (E4M3) KV cache: the four operators of a step, each as
plain torch operations and as the library's call, on seeded inputs.

    tables   paged_batch_tables   block tables, slot maps, positions and offsets from request lengths
    mask     tree_mask            ancestor bits and positions of drafted nodes from parent indices
    attn     attention_tree       attention of the drafted nodes over the cache and their ancestors
    accept   kv_cache_accept      rows of the accepted path moved to consecutive cache positions

A step uses them in this order: the tables give every drafted token its cache slot, the mask its
position (for the rotary embedding) and its ancestors, the cache write stores the nodes' K and V
behind the committed context, the attention reads both, and after verification the accepted nodes'
rows are moved up so that the context is contiguous again.

Lengths are drawn from the case alone (`lens`), so that a case has one size; contents (codes,
trees, block order, accepted paths) come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # One decode step of the benchmark's batch: 64 sequences, contexts U[512, 4096], one token
        # each: a launch-bound call made once per step.
        dict(name="tables_decode_64", op="tables", B=64, ctx_lo=512, ctx_hi=4096, new_lo=1,
             new_hi=1, bs=16, pad=0, lens=7),
        # A drafting batch with odd block size, idle requests and a padded token capacity.
        dict(name="tables_draft_211", op="tables", B=211, ctx_lo=0, ctx_hi=9000, new_lo=0,
             new_hi=33, bs=24, pad=61, lens=8),
        # Prompts of a rollout admitted at once: about a million new tokens.
        dict(name="tables_prompts_256", op="tables", B=256, ctx_lo=0, ctx_hi=64, new_lo=100,
             new_hi=8192, bs=16, pad=0, lens=9),
        # Small dynamic trees of the decode batch.
        dict(name="mask_64x16", op="mask", B=64, n_lo=1, n_hi=16, lens=10),
        # Long drafts, close to chains: deep ancestor lists.
        dict(name="mask_16x1000", op="mask", B=16, n_lo=400, n_hi=1000, lens=11),
        # One user, short context, seven drafted nodes: the latency of the call.
        dict(name="attn_one_short", op="attn", B=1, Hq=32, Hkv=8, D=128, ctx_lo=333, ctx_hi=333,
             n_lo=7, n_hi=7, bs=16, lens=12),
        # The benchmark's decode batch (64 sequences, U[512, 4096] positions) with ragged drafts.
        dict(name="attn_batch_64", op="attn", B=64, Hq=32, Hkv=8, D=128, ctx_lo=512, ctx_hi=4096,
             n_lo=1, n_hi=16, bs=16, lens=7),
        # One long context (past 131072 positions), a wide tree.
        dict(name="attn_long_1", op="attn", B=1, Hq=32, Hkv=8, D=128, ctx_lo=131501, ctx_hi=131501,
             n_lo=61, n_hi=61, bs=64, lens=13),
        # Many nodes per sequence: bound by the tensor cores, not by the cache's bytes.
        dict(name="attn_wide_8", op="attn", B=8, Hq=32, Hkv=8, D=128, ctx_lo=2500, ctx_hi=6000,
             n_lo=300, n_hi=512, bs=16, lens=14),
        # Heads of 64 without sharing, odd block size, short contexts (some empty).
        dict(name="attn_d64_40", op="attn", B=40, Hq=16, Hkv=16, D=64, ctx_lo=0, ctx_hi=2100,
             n_lo=1, n_hi=9, bs=7, lens=15),
        # One layer's cache after verification of the decode batch.
        dict(name="accept_64", op="accept", layers=1, B=64, row=1024, ctx_lo=1, ctx_hi=120,
             n_lo=16, n_hi=16, path=5, bs=16, lens=16),
        # All 36 layers of the requant sweep's model in one call.
        dict(name="accept_36_layers", op="accept", layers=36, B=64, row=1024, ctx_lo=1, ctx_hi=40,
             n_lo=16, n_hi=48, path=9, bs=16, lens=17),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "mask", "attn", "attn", "accept"])
    lens = rng.randrange(1 << 30)
    if op == "tables":
        B = _log_int(rng, 1, 1500)
        hi = _log_int(rng, 1, min(8192, max(1, 1000000 // B)))
        return dict(op=op, B=B, ctx_lo=1, ctx_hi=_log_int(rng, 20, 9000),
                    new_lo=rng.randint(0, hi), new_hi=hi, bs=rng.choice([1, 5, 8, 16, 24, 32, 64]),
                    pad=rng.choice([0, 3, 100]), lens=lens)
    if op == "mask":
        hi = _log_int(rng, 1, 1000)
        return dict(op=op, B=_log_int(rng, 1, max(2, min(300, 16000 // hi))),
                    n_lo=rng.randint(0, hi), n_hi=hi, lens=lens)
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 8])
        D = rng.choice([64, 128])
        hi = _log_int(rng, 1, 512)
        ctx = _log_int(rng, 1, 131072)
        # at most the wide case's products and the long case's positions
        most = min(300, 150000 * 1024 // (Hkv * D * (ctx + hi)), 600000 // (ctx + hi),
                   int(8 * 32 * 400 * 4250 / (Hkv * G * hi * (ctx + hi))))
        B = _log_int(rng, 1, max(1, most))
        if most < 1:
            hi = max(1, 61 * 32 // (Hkv * G))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx,
                    n_lo=rng.randint(1, hi), n_hi=hi, bs=rng.choice([1, 7, 16, 32, 64, 128]),
                    lens=lens)
    n_hi = _log_int(rng, 1, 64)
    return dict(op=op, layers=rng.choice([1, 2, 9, 36]), B=_log_int(rng, 1, 64),
                row=rng.choice([64, 256, 1024]), ctx_lo=0, ctx_hi=40, n_lo=rng.randint(1, n_hi),
                n_hi=n_hi, path=rng.randint(1, 12), bs=rng.choice([1, 7, 16, 64]), lens=lens)


def _lengths(case):
    """(context lengths, new tokens or nodes) of the case's sequences."""
    r = random.Random(case["lens"])
    lo, hi = ("new_lo", "new_hi") if case["op"] == "tables" else ("n_lo", "n_hi")
    n = [r.randint(case[lo], case[hi]) for _ in range(case["B"])]
    ctx = [r.randint(case.get("ctx_lo", 0), case.get("ctx_hi", 0)) for _ in range(case["B"])]
    return ctx, n


def work(case):
    ctx, n = _lengths(case)
    B, total = case["B"], sum(n)
    if case["op"] == "tables":
        bs = case["bs"]
        nb = sum(-(-(c + m) // bs) - -(-c // bs) for c, m in zip(ctx, n))
        return {"bytes": 8 * B + 8 * nb + 8 * B + 16 * (total + case["pad"]) + 8,
                "flops": 0}
    if case["op"] == "mask":
        words = -(-case["n_hi"] // 64)
        return {"bytes": 4 * total + 8 * B + 8 * total * words + 8 * total, "flops": 0}
    if case["op"] == "attn":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        words = -(-case["n_hi"] // 64)
        pos = sum(c + m for c, m in zip(ctx, n))
        blocks = sum(-(-(c + m) // case["bs"]) for c, m in zip(ctx, n))
        return {"bytes": 2 * pos * Hkv * D + 3 * total * Hq * D + 4 * blocks + 8 * B
                + 8 * total * words,
                "flops": 4 * D * Hq * sum(m * (c + 1) for c, m in zip(ctx, n))}
    moved = sum(max(0, min(case["path"], m) - 1) for m in n)
    return {"bytes": 4 * moved * case["row"] * case["layers"] + 4 * B * (case["path"] + 4),
            "flops": 0}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _cuda(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype=dtype, device="cuda")


def _cu(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _trees(n, rng):
    """Parent of each node within its sequence (-1: a child of the context), parents first.  Each
    sequence has its own branching; small ones are near chains."""
    out = []
    for m in n:
        i = np.arange(m)
        br = rng.choice([1.02, 1.5, 2.0, 3.0])
        out.append(np.maximum(-1, np.floor((i - 1) / br).astype(np.int64)
                              - rng.integers(0, 2, m) * (rng.random(m) < 0.3)))
    return np.concatenate(out).astype(np.int32) if out else np.zeros(0, np.int32)


def _mask_bits(parents, cu, words):
    bits = np.zeros((len(parents), words), np.uint64)
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            row = cu[b] + i
            if parents[row] >= 0:
                bits[row] = bits[cu[b] + parents[row]]
            bits[row, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return bits.view(np.int64)


def _block_tables(lengths, bs, rng, spare=5):
    """Blocks dealt to the sequences in random order; unused entries -1."""
    need = [-(-l // bs) for l in lengths]
    width = max(1, max(need))
    perm = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lengths), width), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, len(perm), perm[at:]


def _e4m3(x):
    """Codes and scale amax / 448 of a tensor."""
    s = x.abs().amax() / 448.0
    return (x / s).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    rng = np.random.default_rng([seed, case["lens"]])
    ctx, n = _lengths(case)
    cu = _cu(n)
    total = int(cu[-1])
    if case["op"] == "mask":                 # contexts are values there, not sizes
        ctx = rng.integers(0, 100000, case["B"]).tolist()
    st = dict(case=case, ctx_host=ctx, n_host=n, total=total,
              ctx=_cuda(np.array(ctx), torch.int32), cu=_cuda(cu, torch.int32))
    if case["op"] == "tables":
        bs = case["bs"]
        have = [-(-c // bs) for c in ctx]
        want = [-(-(c + m) // bs) for c, m in zip(ctx, n)]
        fresh = sum(want) - sum(have)
        perm = rng.permutation(sum(want) + 17).astype(np.int32)
        table = np.full((case["B"], max(1, max(want)) + 1), -1, np.int32)
        at = 0
        for b, k in enumerate(have):
            table[b, :k] = perm[at:at + k]
            at += k
        st.update(new=_cuda(np.array(n), torch.int32), table=_cuda(table, torch.int32),
                  free=_cuda(perm[at:], torch.int32), fresh=fresh,
                  free_count=_cuda(np.array([fresh + 11]), torch.int32),
                  capacity=total + case["pad"])
        return st
    parents = _trees(n, rng)
    if case["op"] == "mask":
        st.update(parents=_cuda(parents, torch.int32))
        return st
    if case["op"] == "attn":
        Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
        table, blocks, _ = _block_tables([c + m for c, m in zip(ctx, n)], bs, rng)
        g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 40)))
        slots = blocks * bs
        k = torch.randn((slots, Hkv, D), generator=g, device="cuda")
        loud = torch.from_numpy(rng.permutation(D)[:4].copy()).cuda()
        k[:, :, loud] *= 8.0                              # the outlier channels K shows
        kc, sk = _e4m3(k)
        del k
        vc, sv = _e4m3(torch.randn((slots, Hkv, D), generator=g, device="cuda") * 0.5)
        qc, sq = _e4m3(torch.randn((total, Hq * D), generator=g, device="cuda"))
        words = max(1, -(-case["n_hi"] // 64))
        st.update(q=qc, k=kc.view(slots, Hkv * D), v=vc.view(slots, Hkv * D),
                  scales=torch.stack([sq, sk, sv]).float(), table=_cuda(table, torch.int32),
                  mask=_cuda(_mask_bits(parents, cu, words), torch.int64),
                  longest=max(c + m for c, m in zip(ctx, n)))
        if own:
            import fp8_blockwise_w8a8_b200 as fq
            st["workspace"] = torch.empty(
                max(16, fq.attention_tree_workspace_bytes(case["B"], Hq, Hkv, D, case["n_hi"],
                                                          st["longest"])),
                dtype=torch.uint8, device="cuda")
        return st
    # accept: a path of ascending nodes whose rows are not themselves destinations (breadth-first
    # numbering: the accepted node of each level lies behind the levels above it)
    bs, L, row = case["bs"], case["layers"], case["row"]
    table, blocks, _ = _block_tables([c + m for c, m in zip(ctx, n)], bs, rng)
    slots = blocks * bs
    paths = np.full((case["B"], case["path"]), -1, np.int32)
    plen = np.zeros(case["B"], np.int32)
    for b, m in enumerate(n):
        k = min(case["path"], m)
        rest = np.arange(k, m)
        take = np.sort(rng.permutation(rest)[:max(0, min(k - 1, len(rest)))])
        p = np.concatenate([[0], take]) if m else np.zeros(0)
        paths[b, :len(p)] = p
        plen[b] = len(p)
    g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 40)))
    mk = lambda: torch.randint(0, 256, (L, slots, row), generator=g, device="cuda",
                               dtype=torch.uint8)
    st.update(k=mk(), v=mk(), table=_cuda(table, torch.int32), path=_cuda(paths, torch.int32),
              path_lens=_cuda(plen, torch.int32), plen_host=plen)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _slot_of(table, bs, b, pos):
    blk = table[b, pos // bs].long()
    return torch.where(blk < 0, blk, blk * bs + pos % bs)


def _plain_tables(st):
    bs, total, cap = st["case"]["bs"], st["total"], st["capacity"]
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"]
    B = ctx.numel()
    dev = ctx.device
    cu = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    cu[1:] = new.cumsum(0)
    have, want = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    fresh = want - have
    first = fresh.cumsum(0) - fresh
    k = torch.arange(st["fresh"], device=dev)
    rows = torch.repeat_interleave(torch.arange(B, device=dev), fresh, output_size=st["fresh"])
    table[rows, have[rows] + k - first[rows]] = st["free"][st["free_count"].long() - 1 - k]
    t = torch.arange(total, device=dev)
    req = torch.repeat_interleave(torch.arange(B, device=dev), new, output_size=total)
    pos = ctx[req] + t - cu[req]
    slots = torch.full((cap,), -1, dtype=torch.int64, device=dev)
    positions = torch.zeros(cap, dtype=torch.int64, device=dev)
    slots[:total] = _slot_of(table, bs, req, pos)
    positions[:total] = pos
    return (cu.int(), (ctx + new).int(), slots, positions,
            (st["free_count"] - fresh.sum()).int(), table)


def _plain_mask(st):
    B, N = st["case"]["B"], st["case"]["n_hi"]
    cu, parents = st["cu"].long(), st["parents"].long()
    dev, total = cu.device, st["total"]
    words = -(-N // 64)
    seq = torch.repeat_interleave(torch.arange(B, device=dev), cu[1:] - cu[:-1],
                                  output_size=total)
    node = torch.arange(total, device=dev) - cu[seq]
    # closure of (own bit + parent's bit) by squaring
    m = torch.zeros((B, N, N + 1), device=dev)
    m[seq, node, node] = 1.0
    m[seq, node, torch.where(parents < 0, N, parents)] = 1.0      # column N: the context
    m = m[:, :, :N]
    steps = max(1, math.ceil(math.log2(max(2, N))))
    for _ in range(steps):
        m = (m @ m).clamp_(max=1.0)
    rows = m[seq, node]
    depth = rows.sum(1).long() - 1
    bits = torch.zeros((total, words * 64), dtype=torch.int64, device=dev)
    bits[:, :N] = rows.long()
    bits = bits.view(total, words, 64) << torch.arange(64, device=dev)
    return bits.sum(2), st["ctx"].long()[seq] + depth


def _plain_attn(st):
    case = st["case"]
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    G = Hq // Hkv
    dec = lambda c: c.view(torch.float8_e4m3fn).float()
    scale = st["scales"][0] * st["scales"][1] / math.sqrt(D)
    out = torch.empty((st["total"], Hq * D), dtype=torch.bfloat16, device=st["q"].device)
    shift = torch.arange(64, device=out.device)
    at = 0
    for b, (c, m) in enumerate(zip(st["ctx_host"], st["n_host"])):
        if m == 0:
            continue
        pos = torch.arange(c + m, device=out.device)
        slot = _slot_of(st["table"], bs, b, pos)
        k = dec(st["k"][slot]).view(c + m, Hkv, D).permute(1, 2, 0)
        v = dec(st["v"][slot]).view(c + m, Hkv, D).permute(1, 0, 2)
        q = dec(st["q"][at:at + m]).view(m, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
        z = torch.matmul(q, k).mul_(scale).view(Hkv, m, G, c + m)
        sees = ((st["mask"][at:at + m, :, None] >> shift) & 1).view(m, -1)[:, :m].bool().tril()
        z[..., c:].masked_fill_(~sees[None, :, None, :], float("-inf"))
        z = z.view(Hkv, m * G, c + m)
        z = z.sub_(z.amax(-1, keepdim=True)).exp_()
        den = z.sum(-1, keepdim=True)
        o = torch.matmul(z, v).div_(den).mul_(st["scales"][2])
        out[at:at + m] = (o.view(Hkv, m, G, D).permute(1, 0, 2, 3).reshape(m, Hq * D)
                          .to(torch.bfloat16))
        at += m
    return out


def _plain_accept(st):
    bs = st["case"]["bs"]
    path, plen, ctx = st["path"].long(), st["path_lens"].long(), st["ctx"].long()
    B, P = path.shape
    step = torch.arange(P, device=path.device)
    live = step[None, :] < plen[:, None]
    rows = torch.arange(B, device=path.device)[:, None].expand(B, P)
    # steps behind a path's end copy its first row onto itself
    here = torch.where(live, step[None, :], 0)
    there = torch.where(live, path, 0)
    src = _slot_of(st["table"], bs, rows, ctx[:, None] + there).reshape(-1)
    dst = _slot_of(st["table"], bs, rows, ctx[:, None] + here).reshape(-1)
    for c in (st["k"], st["v"]):
        c[:, dst] = c[:, src]
    return st["k"], st["v"], (ctx + plen).int()


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"tables": _plain_tables, "mask": _plain_mask, "attn": _plain_attn,
                "accept": _plain_accept}[op](state)
    import fp8_blockwise_w8a8_b200 as fq
    if op == "tables":
        out = fq.paged_batch_tables(state["ctx"], state["new"], state["table"], state["free"],
                                    state["free_count"], case["bs"], state["capacity"])
        return (*out, state["table"])
    if op == "mask":
        return fq.tree_mask(state["parents"], state["cu"], case["n_hi"], ctx_lens=state["ctx"])
    if op == "attn":
        return fq.attention_tree(state["q"], state["k"], state["v"], state["scales"],
                                 state["table"], state["ctx"], state["cu"], state["mask"],
                                 case["Hq"], case["Hkv"], case["bs"], case["n_hi"],
                                 state["longest"], workspace=state["workspace"])
    lens = fq.kv_cache_accept(state["k"], state["v"], state["table"], state["ctx"], state["cu"],
                              state["path"], state["path_lens"], case["bs"])
    return state["k"], state["v"], lens


# ---------------------------------------------------------------------------------------------
# definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _decode_table():
    """Value of every E4M3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F is NaN."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        mag = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else -mag if c & 128 else mag
    return torch.from_numpy(v).cuda()


def _exact_attn(case, st):
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    G = Hq // Hkv
    val = _decode_table()
    sq, sk, sv = (x.double() for x in st["scales"])
    out = torch.zeros((st["total"], Hq, D), dtype=torch.float64, device="cuda")
    cu = np.concatenate([[0], np.cumsum(st["n_host"])])
    table = st["table"].cpu().numpy()
    bits = st["mask"].cpu().numpy().view(np.uint64)
    for b in range(case["B"]):
        c, m = st["ctx_host"][b], st["n_host"][b]
        slots = torch.tensor([int(table[b, p // bs]) * bs + p % bs for p in range(c + m)],
                             dtype=torch.int64).cuda()
        see = np.ones((m, c + m), bool)
        j = np.arange(m)
        words = bits[cu[b]:cu[b] + m][:, j // 64]
        see[:, c:] = ((words >> (j % 64).astype(np.uint64)) & np.uint64(1)).astype(bool)
        see[:, c:] &= j[None, :] <= j[:, None]
        see = torch.from_numpy(see).cuda()
        for g in range(Hkv):
            k = val[st["k"][slots, g * D:(g + 1) * D].long()] * sk
            v = val[st["v"][slots, g * D:(g + 1) * D].long()] * sv
            for h in range(g * G, (g + 1) * G):
                q = val[st["q"][cu[b]:cu[b] + m, h * D:(h + 1) * D].long()] * sq
                z = torch.where(see, (q @ k.T) / math.sqrt(D), -math.inf)
                out[cu[b]:cu[b] + m, h] = torch.softmax(z, 1) @ v
    return out.view(st["total"], Hq * D)


def _exact_tables(case, st):
    bs = case["bs"]
    table = st["table"].cpu().numpy().astype(np.int64)
    stack = st["free"].cpu().numpy().tolist()[:int(st["free_count"])]
    slots, positions = [], []
    for b, (c, m) in enumerate(zip(st["ctx_host"], st["n_host"])):
        for k in range(-(-c // bs), -(-(c + m) // bs)):
            table[b, k] = stack.pop()
        pos = np.arange(c, c + m)
        positions.append(pos)
        slots.append(table[b, pos // bs] * bs + pos % bs)
    behind = st["capacity"] - st["total"]
    n = np.array(st["n_host"])
    outs = (np.concatenate([[0], np.cumsum(n)]), np.array(st["ctx_host"]) + n,
            np.concatenate(slots + [np.full(behind, -1)]),
            np.concatenate(positions + [np.zeros(behind)]), np.array([len(stack)]), table)
    return tuple(_cuda(o, torch.int64) for o in outs)


def _exact_mask(case, st):
    parents = st["parents"].cpu().numpy()
    cu = _cu(st["n_host"])
    bits = _mask_bits(parents, cu, -(-case["n_hi"] // 64))
    pos = np.zeros(st["total"], np.int64)
    for b, c in enumerate(st["ctx_host"]):
        for i in range(cu[b], cu[b + 1]):
            pos[i] = c if parents[i] < 0 else pos[cu[b] + parents[i]] + 1
    return _cuda(bits, torch.int64), _cuda(pos, torch.int64)


def _exact_accept(case, st):
    bs = case["bs"]
    table, path = st["table"].cpu().numpy(), st["path"].cpu().numpy()
    src, dst = [], []
    for b, c in enumerate(st["ctx_host"]):
        for i in range(st["plen_host"][b]):
            for where, p in ((src, c + path[b, i]), (dst, c + i)):
                where.append(int(table[b, p // bs]) * bs + int(p) % bs)
    src, dst = _cuda(np.array(src), torch.int64), _cuda(np.array(dst), torch.int64)
    out = [c.index_copy(1, dst, c.index_select(1, src)) for c in (st["k"], st["v"])]
    lens = np.array(st["ctx_host"]) + st["plen_host"]
    return (*out, _cuda(lens, torch.int64))


def exact(case, seed):
    st = prepare(case, seed)
    return {"tables": _exact_tables, "mask": _exact_mask, "attn": _exact_attn,
            "accept": _exact_accept}[case["op"]](case, st)
