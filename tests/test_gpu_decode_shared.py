"""Paged decode of groups that share their first pages against its definition in 64 bits (bounds in
paged_ref.check).  Every slot that no query may see holds NaN, and so do the shared entries of all but a
group's first table row."""
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def wide(H, Hkv, d, S, shared, ctx):
    """Spare columns that bring the repeated reads, by the table's capacity, past what is left to L2 (180 MB at most)."""
    B = len(ctx)
    return 1 + int(1.9e8 / (2 * max(1, B - B // S) * Hkv * 16 * d))


def widest(H, Hkv, d, S, shared, ctx):
    """Spare columns that keep them well below it, but for few rows end the form whose splits are a cluster."""
    B = len(ctx)
    used = max(max((c + 15) // 16 for c in ctx), max(shared))
    return max(1, min(2100, int(7.5e7 / (4 * max(1, B - B // S) * Hkv * 16 * d)) - used))


def make(H, Hkv, d, S, shared, ctx, fp8, seed, spare=1):
    """shared: pages of each group; ctx: tokens of each sequence.  Returns the call's tensors and full tables."""
    G, B = len(shared), len(ctx)
    assert B == G * S
    own = [max(0, (c + 15) // 16 - shared[b // S]) for b, c in enumerate(ctx)]
    width = max(shared[b // S] + own[b] for b in range(B)) + spare
    total = sum(shared) + sum(own)
    k, v, nan = R.cache(total, Hkv, d, seed, fp8)
    g = torch.Generator().manual_seed(seed + 1)
    perm = torch.randperm(total, generator=g).to(torch.int32)
    full = torch.full((B, width), nan, dtype=torch.int32)
    at = 0
    for i in range(G):
        full[i * S:(i + 1) * S, :shared[i]] = perm[at:at + shared[i]]
        at += shared[i]
        longest = max(ctx[i * S:(i + 1) * S])
        for p in range(shared[i]):  # shared slots past every sequence of the group
            if longest < (p + 1) * 16:
                R.poison(k, v, int(full[i * S, p]), max(0, longest - p * 16), 16, fp8)
    for b in range(B):
        n = shared[b // S]
        full[b, n:n + own[b]] = perm[at:at + own[b]]
        at += own[b]
        if own[b] and ctx[b] % 16:
            R.poison(k, v, int(full[b, n + own[b] - 1]), ctx[b] % 16, 16, fp8)
    table = full.clone()
    for b in range(B):
        if b % S:
            table[b, :shared[b // S]] = -1  # read from the group's first row alone
    q = (torch.randn(B, H, d, generator=g) * 2).to(torch.bfloat16)
    return dict(q=q, k=k, v=v, table=table, full=full, ctx=torch.tensor(ctx, dtype=torch.int32),
                shared=torch.tensor(shared, dtype=torch.int32), S=S)


def run(lib, x, fp8, **kw):
    a = [x[n].cuda() for n in ("q", "k", "v")]
    b = [x[n].cuda() for n in ("table", "ctx", "shared")]
    if fp8:
        return lib.paged_attn_decode_shared_fp8(*a, 0.02, 0.02, *b, x["S"], **kw)
    return lib.paged_attn_decode_shared(*a, *b, x["S"], **kw)


CASES = [  # H, Hkv, d, S, shared pages per group, contexts
    (1, 1, 32, 1, [2], [40]),                                     # a group of one
    (4, 4, 64, 2, [4, 0], [64, 65, 16, 0]),                       # no own pages, nothing shared, an empty place
    (12, 12, 64, 4, [40], [700, 641, 648, 656]),
    (14, 2, 80, 3, [5, 9], [100, 200, 81, 144, 500, 150]),        # seven heads per key/value head
    (6, 2, 96, 5, [33], [530, 7, 0, 528, 1000]),                  # contexts that end inside the shared pages
    (32, 8, 128, 33, [64], [1024 + 13 * i for i in range(33)]),   # more rows than one tile
    (16, 1, 128, 20, [100], [1600 + (i * 37) % 300 for i in range(20)]),   # more than two tiles, 16 heads
    (8, 1, 32, 40, [17, 3], [272 + i for i in range(40)] + [48 + 2 * i for i in range(40)]),
    (24, 1, 64, 2, [6], [130, 97]),                               # 24 heads: two row groups
    (130, 1, 32, 2, [3], [60, 100]),                              # more heads than a tile has rows
    (8, 8, 128, 2, [1], [5, 12]),                                 # all of it inside the first shared page
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("spare", [None, widest, wide], ids=["per_sequence", "per_sequence_wide", "per_group"])
@pytest.mark.parametrize("case", CASES, ids=[f"H{c[0]}kv{c[1]}d{c[2]}S{c[3]}G{len(c[4])}" for c in CASES])
def test_matches_the_definition(lib, case, spare, fp8):
    H, Hkv, d, S, shared, ctx = case
    x = make(H, Hkv, d, S, shared, ctx, fp8, 3, spare=spare(H, Hkv, d, S, shared, ctx) if spare else 1)
    B = len(ctx)
    o = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), float("nan"), device="cuda")
    run(lib, x, fp8, out=o, lse=lse)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    R.check(o.cpu(), lse.cpu(), *R.decode(x["q"], x["k"], x["v"], x["full"], ctx, d ** -0.5, fp8))


@pytest.mark.parametrize("once", [False, True], ids=["per_sequence", "per_group"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_unmapped_shared_pages_and_clamped_counts(lib, fp8, once):
    x = make(4, 2, 64, 2, [10, 3, 2], [200, 190, 60, 77, 0, 0], fp8, 4, spare=24000 if once else 1)
    for t in (x["table"], x["full"]):
        t[0:2, 4] = -1
        t[2:4, 0] = 10**6
    x["shared"] = torch.tensor([10, 3, -4], dtype=torch.int32)
    out = run(lib, x, fp8)
    R.check(out[0].cpu(), out[1].cpu(), *R.decode(x["q"], x["k"], x["v"], x["full"], x["ctx"].tolist(), 64 ** -0.5, fp8))
    # more shared pages than the table has columns, contexts longer than the table
    y = make(4, 2, 64, 2, [4], [64, 64], fp8, 5, spare=0)
    y["shared"] = torch.tensor([10**6], dtype=torch.int32)
    y["ctx"] = torch.tensor([10**9, 30], dtype=torch.int32)
    out = run(lib, y, fp8)
    R.check(out[0].cpu(), out[1].cpu(), *R.decode(y["q"], y["k"], y["v"], y["full"], y["ctx"].tolist(), 64 ** -0.5, fp8))


@pytest.mark.parametrize("once", [False, True], ids=["per_sequence", "per_group"])
def test_other_stream_graph_and_repeats(lib, once):
    x = make(8, 2, 128, 4, [30, 12], [500 + 9 * i for i in range(4)] + [200 + 30 * i for i in range(4)], False, 6,
             spare=6000 if once else 1)
    want = run(lib, x, False)
    a = [x[n].cuda() for n in ("q", "k", "v", "table", "ctx", "shared")]
    need = lib.paged_attn_decode_shared_workspace_size(8, 8, 2, 128, x["table"].shape[1], 4)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):  # back to back on one workspace
        got = lib.paged_attn_decode_shared(*a, 4, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = lib.paged_attn_decode_shared(*a, 4)
        two = lib.paged_attn_decode_shared(*a, 4)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got in (one, two):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_prompt_once_then_samples(lib):
    """As it is used: a prompt goes into shared pages, samples append their own tokens with the rotation, and
    the shared decode gives what a decode of each sequence alone gives."""
    H, Hkv, d, S = 8, 2, 64, 3
    prompt, steps = 64, 5
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    kp, vp = (torch.full((4 + S, Hkv, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[0, 1, 2, 3, 4 + i] for i in range(S)], dtype=torch.int32, device="cuda")
    a = torch.arange(128, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cs = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.paged_kv_append_rope(None, rnd(1, Hkv, prompt, d), rnd(1, Hkv, prompt, d), kp, vp, cs, table[:1], zero)
    shared = torch.tensor([prompt // 16], dtype=torch.int32, device="cuda")
    for i in range(steps):
        start = torch.full((S,), prompt + i, dtype=torch.int32, device="cuda")
        q = lib.paged_kv_append_rope(rnd(S, H, 1, d), rnd(S, Hkv, 1, d), rnd(S, Hkv, 1, d), kp, vp, cs, table, start)
        ctx = start + 1
        o, lse = lib.paged_attn_decode_shared(q.view(S, H, d), kp, vp, table, ctx, shared, S)
        want = R.decode(q.view(S, H, d).cpu(), kp.cpu(), vp.cpu(), table.cpu(), ctx.tolist(), d ** -0.5)
        R.check(o.cpu(), lse.cpu(), *want)
