"""Paged decode with modified scores against its definition in 64 bits (bounds in paged_ref.check).  Every
slot that a query must not see holds NaN."""
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


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])


def make(B, H, Hkv, d, ctx, fp8, seed, begin=None, spare=2):
    width = max(1, max((c + 15) // 16 for c in ctx)) + spare
    per = [(c + 15) // 16 for c in ctx]
    k, v, nan = R.cache(sum(per), Hkv, d, seed, fp8)
    g = torch.Generator().manual_seed(seed + 1)
    perm = torch.randperm(sum(per), generator=g)
    table = torch.full((B, width), nan, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
        if ctx[b] % 16:
            R.poison(k, v, int(table[b, n - 1]), ctx[b] % 16, 16, fp8)
        if begin is not None and 0 < begin[b] < ctx[b]:
            table[b, :begin[b] // 16] = nan
            R.poison(k, v, int(table[b, begin[b] // 16]), 0, begin[b] % 16, fp8)
    q = (torch.randn(B, H, d, generator=g) * 2).to(torch.bfloat16)
    return q, k, v, table, torch.tensor(ctx, dtype=torch.int32)


def run(lib, x, fp8, **kw):
    q, k, v, table, ctx = (t.cuda() for t in x)
    kw = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in kw.items()}
    if fp8:
        return lib.paged_attn_decode_scoremod_fp8(q, k, v, 0.02, 0.02, table, ctx, **kw)
    return lib.paged_attn_decode_scoremod(q, k, v, table, ctx, **kw)


# A narrow table is cut into clusters of CTAs, which merge among themselves; one this wide into splits that go
# through the workspace.
WIDE = 2100
FORMS = dict(argvalues=[2, WIDE], ids=["cluster", "workspace"])

SHAPES = [  # B, H, Hkv, d, contexts
    (1, 1, 1, 32, [1]), (4, 4, 4, 64, [0, 16, 17, 1025]), (3, 14, 2, 80, [333, 15, 2000]), (2, 12, 1, 96, [1024, 70]),
    (2, 16, 1, 128, [3000, 129]), (2, 40, 2, 128, [513, 900]), (3, 32, 8, 128, [4097, 1, 640]), (1, 6, 2, 32, [2600]),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("mod", [(0.0, False, 0), (5.0, False, 0), (0.0, True, 100), (30.0, True, 33)],
                         ids=["plain", "cap5", "bias_window", "cap30_bias_window"])
@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=[f"B{s[0]}H{s[1]}kv{s[2]}d{s[3]}" for s in SHAPES])
def test_matches_the_definition(lib, shape, spare, mod, fp8):
    B, H, Hkv, d, ctx = shape
    cap, bias, window = mod
    begin = [c - window for c in ctx] if window else None
    x = make(B, H, Hkv, d, ctx, fp8, 3, begin, spare)
    sl = slopes_of(H) if bias else None
    kb = None if begin is None else torch.tensor(begin, dtype=torch.int32)
    o = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), float("nan"), device="cuda")
    run(lib, x, fp8, softcap=cap, alibi_slopes=sl, key_begin=kb, out=o, lse=lse)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    R.check(o.cpu(), lse.cpu(), *R.decode(x[0], x[1], x[2], x[3], ctx, d ** -0.5, fp8, cap, sl, begin))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("spare", [0, WIDE], ids=["cluster", "workspace"])
def test_unmapped_pages_and_odd_intervals(lib, fp8, spare):
    ctx = [200, 300, 64, 500, 5000, 50]
    begin = [200, 2**31 - 1, -5, 250, 10, 50]  # nothing left, nothing left, all, a page's middle, nothing left
    x = make(6, 4, 2, 64, ctx, fp8, 5, spare=spare)
    x[3][0, 1], x[3][3, 20], x[3][2, 0] = -1, 10**6, -7
    x[3][5, :] = x[1].shape[0]  # no page mapped at all
    out = run(lib, x, fp8, softcap=10.0, alibi_slopes=slopes_of(4), key_begin=torch.tensor(begin, dtype=torch.int32))
    R.check(out[0].cpu(), out[1].cpu(), *R.decode(x[0], x[1], x[2], x[3], [int(c) for c in x[4]], 64 ** -0.5, fp8, 10.0,
                                                  slopes_of(4), begin))


def test_plain_call_agrees_with_the_plain_decode(lib):
    x = make(4, 8, 2, 128, [700, 30, 1, 1999], False, 6)
    a = run(lib, x, False)
    q, k, v, table, ctx = (t.cuda() for t in x)
    b = lib.paged_attn_decode_gqa(q, k, v, table, ctx)
    # two evaluations of the same definition, each within its bound: a rounding of the weights and of O apart
    assert (a[0].double() - b[0].double()).abs().max() <= 2 * 2.0 ** -7 * b[0].double().abs().max()
    assert (a[1] - b[1]).abs().max() <= 2e-4


def test_huge_queries_over_e4m3_pages(lib):
    # queries past f16's range: rounded to f16 after a power of two, which returns in the scale
    x = list(make(2, 4, 2, 64, [40, 90], True, 7))
    x[0] = (x[0].float() * 2.0 ** 20).to(torch.bfloat16)
    scale = 64 ** -0.5 * 2.0 ** -20
    out = run(lib, x, True, scale=scale, softcap=20.0)
    R.check(out[0].cpu(), out[1].cpu(), *R.decode(x[0], x[1], x[2], x[3], [40, 90], scale, True, 20.0))


def test_many_rows_with_few_splits(lib):
    # 64 x 8 rows of CTAs: one CTA each over an e4m3 cache, two per row at half the batch
    for B in (32, 64):
        ctx = [(b * 97) % 1200 for b in range(B)]
        x = make(B, 8, 8, 32, ctx, True, 9)
        out = run(lib, x, True, softcap=20.0)
        R.check(out[0].cpu(), out[1].cpu(), *R.decode(x[0], x[1], x[2], x[3], ctx, 32 ** -0.5, True, 20.0))


@pytest.mark.parametrize("spare", **FORMS)
def test_other_stream_graph_and_workspace(lib, spare):
    x = make(3, 8, 2, 64, [300, 17, 1500], False, 8, spare=spare)
    want = run(lib, x, False, softcap=20.0)
    side = torch.cuda.Stream()
    q, k, v, table, ctx = (t.cuda() for t in x)
    need = lib.paged_attn_decode_scoremod_workspace_size(3, 8, 2, 64, table.shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = lib.paged_attn_decode_scoremod(q, k, v, table, ctx, softcap=20.0, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(lib.AttnError):
        lib.paged_attn_decode_scoremod(q, k, v, table, ctx, softcap=20.0, workspace=ws[:need - 16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = lib.paged_attn_decode_scoremod(q, k, v, table, ctx, softcap=20.0)
    graph.replay()
    ctx.copy_(torch.tensor([100, 16, 1501], dtype=torch.int32))  # lengths are read at each replay
    graph.replay()
    torch.cuda.synchronize()
    want = lib.paged_attn_decode_scoremod(q, k, v, table, ctx, softcap=20.0)
    # sequence 2's 1501st token is a slot of NaN in this cache: the others
    assert torch.equal(cap[0][:2], want[0][:2]) and torch.equal(cap[1][:2], want[1][:2])
