"""Page tables and reference counts by their definition, in plain Python, and random states for the tests."""
import random

import torch


def fork(table, ctx, parents, ref, P):
    W, out, lens = len(table[0]), [], []
    for b, p in enumerate(parents):
        if not 0 <= p < len(table):
            out.append([-1] * W)
            lens.append(0)
            continue
        n = -(-min(max(ctx[p], 0), 16 * W) // 16)
        out.append(list(table[p]) if p == b else table[p][:n] + [-1] * (W - n))
        lens.append(ctx[p])
    ref = list(ref)
    for t, sign in ((out, 1), (table, -1)):
        for row in t:
            for e in row:
                if 0 <= e < P:
                    ref[e] += sign
    return out, lens, ref


def reserve(table, ctx, new, ref, P):
    W, start = len(table[0]), list(ref)
    free = [i for i in range(P) if start[i] <= 0]
    table, ref = [list(r) for r in table], list(ref)
    reserved, src, dst, asked = [], [], [], 0
    for b, row in enumerate(table):
        n = min(max(ctx[b], 0), 16 * W)
        to, s, d, got = -(-(n + new[b]) // 16), -1, -1, 0
        if new[b] > 0 and to <= W:
            want = [c for c in range(n // 16, to) if not 0 <= row[c] < P or start[row[c]] > 1]
            asked += len(want)
            if not want or asked <= len(free):
                got = new[b]
                for c, page in zip(want, free[asked - len(want):]):
                    old, row[c] = row[c], page
                    ref[page] = 1
                    if 0 <= old < P:
                        ref[old] -= 1
                        if c == n // 16 and n % 16:
                            s, d = old, page
        reserved.append(got)
        src.append(s)
        dst.append(d)
    return table, ref, reserved, src, dst


def compact(table, ref, P):
    live = [i for i in range(P) if ref[i] > 0]
    L = len(live)
    src, dst = [i for i in live if i >= L], [i for i in range(L) if ref[i] <= 0]
    to = {i: i for i in live if i < L} | dict(zip(src, dst))
    out = [[to.get(e, -1) for e in row] for row in table]
    counts = [0] * P
    for i, j in to.items():
        counts[j] = ref[i]
    return out, counts, src + [-1] * (P - len(src)), dst + [-1] * (P - len(dst)), len(src)


def state(B, W, P, seed, fill=0.6, share=0.5):
    """A table whose rows share prefixes and tails, its tokens and its counts."""
    r = random.Random(seed)
    ids = list(range(P))
    r.shuffle(ids)
    table, ctx = [], []
    for b in range(B):
        n = r.randint(0, int(16 * W * fill))
        pages = -(-n // 16)
        row = []
        if table and r.random() < share:
            other = r.randrange(len(table))
            k = r.randint(0, min(pages, -(-ctx[other] // 16)))
            row = table[other][:k]
        while len(row) < pages and ids:
            row.append(ids.pop())
        n = min(n, 16 * len(row))
        table.append(row + [-1] * (W - len(row)))
        ctx.append(n)
    ref = [0] * P
    for row in table:
        for e in row:
            if e >= 0:
                ref[e] += 1
    return table, ctx, ref


def i32(x):
    return torch.tensor(x, dtype=torch.int32)
