"""Forking, reserving, compacting and copying of pages against their definition (pages_ref), whole numbers and copies bit for
bit; and all of it as a serving loop uses it."""
import random

import pytest
import torch

import pages_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def dev(*xs):
    return [R.i32(x).cuda() for x in xs]


def same(got, want):
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), R.i32(w).view(g.shape)), (g, w)


SIZES = [(1, 1, 1), (1, 3, 2), (3, 5, 17), (16, 40, 333), (100, 33, 3001), (7, 200, 9000), (300, 20, 70001), (2000, 3, 5000)]  # B, W, P


@pytest.mark.parametrize("B, W, P", SIZES)
def test_fork(lib, B, W, P):
    for seed, Bo in ((1, B), (2, B + 3), (3, max(1, B // 2))):
        table, ctx, ref = R.state(B, W, P, seed)
        r = random.Random(seed)
        parents = [r.choice((b, r.randrange(B), r.randrange(B), -1, B + 5)) for b in range(Bo)]
        ctx[0] += 16 * W  # past the table's capacity: clamped
        ref[r.randrange(P)] += 1  # a page that the caller holds
        t, c, p, n = dev(table, ctx, parents, ref)
        want = R.fork(table, ctx, parents, ref, P)
        same(lib.paged_kv_fork(t, c, p, n), want)
        out = lib.paged_kv_fork(t, c, p, n, ref_counts_out=n)  # the counts in place
        assert out[2] is n
        same(out, want)
        assert torch.equal(t.cpu(), R.i32(table))


@pytest.mark.parametrize("B, W, P", SIZES)
def test_reserve(lib, B, W, P):
    for seed in range(4):
        table, ctx, ref = R.state(B, W, P, seed, fill=(0.2, 0.6, 0.95, 1.0)[seed])
        r = random.Random(seed)
        new = [r.choice((0, 1, 1, 1, -3, r.randint(1, 40), 16 * W, 2**31 - 1)) for _ in range(B)]
        if seed == 2:
            table[0][0] = P + 7  # outside the pool: names no page
        if seed == 3:
            ref[0], ctx[-1] = ref[0] - (ref[0] <= 0), -5  # a count below zero is free too; a negative length is 0
        t, c, a, n = dev(table, ctx, new, ref)
        want = R.reserve(table, ctx, new, ref, P)
        same(lib.paged_kv_reserve(t, c, a, n), want)
        assert torch.equal(t.cpu(), R.i32(table)) and torch.equal(n.cpu(), R.i32(ref))
        ws = torch.full((lib.paged_kv_reserve_workspace_size(B, P),), 255, dtype=torch.uint8, device="cuda")
        out = lib.paged_kv_reserve(t, c, a, n, page_table_out=t, ref_counts_out=n, workspace=ws)  # in place
        assert out[0] is t and out[1] is n
        same(out, want)


def test_reserve_when_many_share_the_last_page(lib):
    # 50 samples of one prompt of 21 tokens: each gets a copy of its own, and the prompt's page ends with a count of 0
    table, ctx, ref = [[3, 5] + [-1] * 2] * 50, [21] * 50, [0] * 64
    ref[3] = ref[5] = 50
    want = R.reserve(table, ctx, [1] * 50, ref, 64)
    same(lib.paged_kv_reserve(*dev(table, ctx, [1] * 50, ref)), want)
    assert want[1][5] == 0 and want[1][3] == 50 and all(s == 5 for s in want[3])


@pytest.mark.parametrize("B, W, P", SIZES)
def test_compact(lib, B, W, P):
    for seed, fill in ((1, 0.3), (2, 1.0)):
        table, ctx, ref = R.state(B, W, P, seed, fill)
        r = random.Random(seed)
        ref[r.randrange(P)] += 1  # held by the caller alone, or by one more
        if seed == 2:
            table[0][0] = r.choice((-9, P))
        t, n = dev(table, ref)
        want = R.compact(table, ref, P)
        same(lib.paged_kv_compact(t, n), want)
        out = lib.paged_kv_compact(t, n, page_table_out=t)
        assert out[0] is t
        same(out, want)


def test_compact_of_an_empty_and_a_full_pool(lib):
    for ref in ([0] * 100, [1] * 100, [0] * 99 + [2], [2] + [0] * 99):
        table = [[99, 0, -1]]
        same(lib.paged_kv_compact(*dev(table, ref)), R.compact(table, ref, 100))


@pytest.mark.parametrize("shape, dtype", [((2, 16, 32), torch.bfloat16), ((1, 9 * 32), torch.uint8), ((8, 16, 128), torch.bfloat16),
                                          ((3, 9 * 80), torch.uint8), ((16,), torch.uint8), ((5, 16, 96), torch.uint8)])
@pytest.mark.parametrize("pools", [1, 2, 300])
def test_copy_pages(lib, shape, dtype, pools):
    P = 40
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randint(0, 256, (P, *shape), generator=g, device="cuda").to(dtype) for _ in range(pools)]
    perm = torch.randperm(P, generator=g, device="cuda").int()
    src, dst = perm[:17].clone(), perm[17:34].clone()
    src[3], dst[5], src[7], dst[9] = -1, P, 2**31 - 1, -2**31
    want = [t.clone() for t in x]
    ok = (src >= 0) & (src < P) & (dst >= 0) & (dst < P)
    for t in want:
        t[dst[ok].long()] = t[src[ok].long()]
    y = [t.clone() for t in x]
    lib.paged_kv_copy_pages(x, src, dst)
    assert all(torch.equal(a, b) for a, b in zip(x, want))
    for n in (0, 4, 100, -1):
        z = [t.clone() for t in y]
        lib.paged_kv_copy_pages(tuple(z), src, dst, count=R.i32([n]).cuda())
        k = min(max(n, 0), 17)
        want = [t.clone() for t in y]
        for t in want:
            t[dst[:k][ok[:k]].long()] = t[src[:k][ok[:k]].long()]
        assert all(torch.equal(a, b) for a, b in zip(z, want)), n


def test_copy_past_32_bit_offsets(lib):
    P = (5 << 30) // (1 << 20)
    x = torch.zeros(P, 1 << 20, dtype=torch.uint8, device="cuda")
    x[P - 2] = 7
    x[1] = 9
    lib.paged_kv_copy_pages([x], *dev([P - 2, 1], [0, P - 1]))
    assert (x[0] == 7).all() and (x[P - 1] == 9).all() and int(x[2:P - 2].max()) == 0


def test_refusals(lib):
    t, c, p, n = dev([[0, -1]], [5], [0], [1, 0])
    with pytest.raises(lib.AttnError):
        lib.paged_kv_fork(t, c, p, n, page_table_out=t)
    with pytest.raises(lib.AttnError):
        lib.paged_kv_compact(t, n, ref_counts_out=n)
    with pytest.raises(lib.AttnError):
        lib.paged_kv_reserve(t, c, p, n, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    pools = [torch.zeros(2, 8, device="cuda"), torch.zeros(2, 16, device="cuda")]
    for bad in (pools, [pools[0], pools[0][:1]], [], [pools[0], pools[0].cpu()], [pools[0].t()]):
        with pytest.raises(ValueError):
            lib.paged_kv_copy_pages(bad, c, p)
    with pytest.raises(lib.AttnError):
        lib.paged_kv_copy_pages([torch.zeros(2, 3, device="cuda")], c, p)  # pages of 12 bytes


def test_other_stream_and_captured_graph(lib):
    P, B, W = 3000, 40, 30
    table, ctx, ref = R.state(B, W, P, 5)
    t, c, n, p, a = dev(table, ctx, ref, [b // 2 for b in range(B)], [1] * B)
    pool = torch.randint(0, 256, (P, 64), dtype=torch.uint8, device="cuda")

    def step(pool, **kw):
        t2, c2, n2 = lib.paged_kv_fork(t, c, p, n, **kw)
        t3, n3, got, src, dst = lib.paged_kv_reserve(t2, c2, a, n2, **kw)
        lib.paged_kv_copy_pages([pool], src, dst, **kw)
        t4, n4, src, dst, count = lib.paged_kv_compact(t3, n3, **kw)
        lib.paged_kv_copy_pages([pool], src, dst, count, **kw)
        return t4, n4, got, src, dst, count

    one, two = pool.clone(), pool.clone()
    want = step(one)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(two, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(one, two)
    three = pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step(three)
    for seed in (5, 6):  # another state in the same memory
        table, ctx, ref = R.state(B, W, P, seed)
        for x, y in ((t, table), (c, ctx), (n, ref)):
            x.copy_(R.i32(y))
        three.copy_(pool)
        graph.replay()
        one = pool.clone()
        assert all(torch.equal(x, y) for x, y in zip(cap, step(one))) and torch.equal(one, three)


def test_serving_loop_over_a_four_bit_cache(lib):
    """Prompts with images come in, are sampled several times, some samples end, the pool is compacted, and every step's
    attention is that over a cache in which each sequence has pages of its own, never forked or moved."""
    import fp4_ref as F
    import paged_ref as PR
    torch.manual_seed(3)
    H, Hkv, d, P, W, ks, vs = 4, 2, 64, 64, 8, 0.01, 0.02
    pools = [torch.zeros(P, Hkv, 9 * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    lone = [torch.zeros(16 * W, Hkv, 9 * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    a = torch.arange(200)[:, None] * 100.0 ** (-torch.arange(0, d, 2) / d)
    cs, pair = torch.cat([a.cos(), a.sin()], 1).float().cuda(), bytes(i % 3 for i in range(d // 2))
    table, ctx, ref = torch.full((2, W), -1, dtype=torch.int32).cuda(), R.i32([0, 0]).cuda(), torch.zeros(P, dtype=torch.int32).cuda()
    rows = [[], []]  # each sequence's tokens: (k, v, positions)

    def add(new):
        nonlocal table, ref, ctx
        N, B = max(new), len(new)
        q = torch.randn(B, N, H, d, device="cuda").to(torch.bfloat16).transpose(1, 2)
        k, v = (torch.randn(B, N, Hkv, d, device="cuda").to(torch.bfloat16).transpose(1, 2) for _ in range(2))
        pos = torch.randint(0, 200, (3, B, N), dtype=torch.int32, device="cuda")
        table, ref, got, src, dst = lib.paged_kv_reserve(table, ctx, R.i32(new).cuda(), ref)
        assert got.tolist() == new
        lib.paged_kv_copy_pages(pools, src, dst)
        q = lib.paged_kv_append_fp4(q, k, v, *pools, ks, vs, table, ctx, cos_sin=cs, positions=pos, pair_axis=pair, new_lens=got)
        for b, n in enumerate(new):
            rows[b] = rows[b] + [(k[b, :, t], v[b, :, t], pos[:, b, t]) for t in range(n)]
        ctx = ctx + got
        return q

    def check(q):
        """The last new token's attention; the oracle's cache is built from the rows' own tokens."""
        B = len(rows)
        own = torch.arange(B * W, dtype=torch.int32, device="cuda").view(B, W)
        for b, r in enumerate(rows):
            if r:
                k, v = (torch.stack([x[i] for x in r], 1)[None] for i in range(2))
                pos = torch.stack([x[2] for x in r], 1)[:, None].contiguous()
                lib.paged_kv_append_fp4(None, k, v, *lone, ks, vs, own[b:b + 1].contiguous(), torch.zeros(1, dtype=torch.int32).cuda(),
                                        cos_sin=cs, positions=pos, pair_axis=pair)
        o, lse = lib.paged_attn_decode_fp4(q, *pools, ks, vs, table, ctx)
        o2, lse2 = lib.paged_attn_decode_fp4(q, *lone, ks, vs, own, ctx)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        want = PR.decode(q.cpu(), F.read(lone[0].cpu(), False) * ks, F.read(lone[1].cpu(), True) * vs, own.cpu(), ctx.tolist(), d ** -0.5)
        PR.check(o.cpu(), lse.cpu(), *want)
        count = torch.bincount(table[table >= 0].long(), minlength=P)
        assert torch.equal(count.int(), ref)

    q = add([37, 20])
    check(torch.stack([q[0, :, 36], q[1, :, 19]]))
    # the chunked prefill over the cache: its pages as bf16, and the paged prefill over those
    bits = lib.paged_kv_unpack_fp4(*pools, ks, vs, table.flatten())
    places = torch.where(table >= 0, torch.arange(2 * W, device="cuda", dtype=torch.int32).view(2, W), -1)
    last = torch.stack([q[0, :, 33:37], q[1, :, 16:20]])
    o, lse = lib.paged_attn_prefill(last.contiguous(), *bits, places, ctx, True)
    kk, vv = F.read(pools[0].cpu(), False) * ks, F.read(pools[1].cpu(), True) * vs
    for i in range(4):
        want = PR.decode(last[:, :, i].cpu(), kk, vv, table.cpu(), (ctx - 3 + i).tolist(), d ** -0.5)
        # K and V are rounded to bf16 on the way (2^-9 of each here too): scores by that of |s| <= about 8, so weights by 2^-6
        assert (o[:, :, i].cpu().double() - want[0]).abs().max() <= (2.0 ** -6 + 2.0 ** -7) * want[2].max() + 2.0 ** -8
    # three samples of each
    table, ctx, ref = lib.paged_kv_fork(table, ctx, R.i32([0, 0, 0, 1, 1, 1]).cuda(), ref)
    rows = [list(rows[i]) for i in (0, 0, 0, 1, 1, 1)]
    for step in range(20):
        check(add([1] * len(rows))[:, :, 0])
        if step == 6:  # beams: rows continue others, one ends
            par = [0, 2, 2, 5, 4, -1]
            table, ctx, ref = lib.paged_kv_fork(table, ctx, R.i32(par).cuda(), ref)
            rows = [list(rows[p]) if p >= 0 else [] for p in par]
        if step == 12:
            table, ref, src, dst, n = lib.paged_kv_compact(table, ref)
            lib.paged_kv_copy_pages(pools, src, dst, n)
            live = int((ref > 0).sum())
            assert int(table.max()) == live - 1
            for p in pools:
                p[live:] = 0x7F  # the pool's end is free for anything
    assert lib.attn_check_device_status() == 0


@pytest.mark.parametrize("B, W, P", [(128, 300, 20000), (40, 1000, 70001), (3, 20011, 9000), (1100, 40, 6000)])
def test_large_tables(lib, B, W, P):
    # tables past what one cluster copies, with pools of both kinds, and more rows than one tile of sums
    test_fork(lib, B, W, P)
    test_reserve(lib, B, W, P)
    test_compact(lib, B, W, P)


@pytest.mark.parametrize("B, W, P", [(128, 300, 20000), (8, 40, 400)])
def test_branches_captured_and_on_two_streams(lib, B, W, P):
    # a fork, a reservation, the copies and a compaction in one graph, replayed on new parents while another user runs the same
    def make(seed):
        table, ctx, ref = R.state(B, W, P, seed, fill=0.6)
        r = random.Random(seed)
        return table, ctx, ref, [r.choice((b, r.randrange(B), -1)) for b in range(B)]

    def want(table, ctx, ref, parents, pool):
        table, ctx, ref = R.fork(table, ctx, parents, ref, P)
        table, ref, got, src, dst = R.reserve(table, ctx, [1] * B, ref, P)
        for s, d in zip(src, dst):
            if s >= 0:
                pool[d] = pool[s]
        table, ref, src, dst, n = R.compact(table, ref, P)
        pool = list(pool)
        for s, d in zip(src, dst):
            if s >= 0:
                pool[d] = pool[s]
        return table, ctx, ref, got, pool

    def run(t, c, n, p, one, pool):
        t, c, n = lib.paged_kv_fork(t, c, p, n)
        t, n, got, src, dst = lib.paged_kv_reserve(t, c, one, n)
        lib.paged_kv_copy_pages([pool], src, dst)
        t, n, src, dst, count = lib.paged_kv_compact(t, n)
        lib.paged_kv_copy_pages([pool], src, dst, count=count)
        return t, c, n, got

    def check(got, pool, state):
        w = want(*state, list(range(P)))
        same(got, w[:4])
        live = torch.tensor([r > 0 for r in w[2]])
        assert torch.equal(pool[:, 0].cpu()[live], R.i32(w[4])[live])

    fresh = torch.arange(P, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4)
    states = [make(s) for s in (1, 2, 3)]
    dev_states = [dev(t, c, n, p) for t, c, n, p in states]
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    inputs, pool = [x.clone() for x in dev_states[0]], fresh.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*inputs, one, pool)
    side = torch.cuda.Stream()
    other = fresh.clone()
    torch.cuda.synchronize()
    for state, new in zip(states[:2], dev_states[:2]):
        for x, y in zip(inputs, new):
            x.copy_(y)
        pool.copy_(fresh)
        other.copy_(fresh)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            beside = run(*dev_states[2], one, other)
        torch.cuda.synchronize()
        check(out, pool, state)
        check(beside, other, states[2])
