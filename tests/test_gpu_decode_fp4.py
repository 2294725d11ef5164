"""Paged decode over the 4-bit cache against its definition in 64 bits (bounds in paged_ref.check: the codes' values are
exact in f16, queries and weights are rounded to it once).  Every slot that a query must not see holds NaN scales."""
import pytest
import torch

import fp4_ref as F
import paged_ref as R
from test_gpu_decode_scoremod import FORMS, SHAPES, WIDE, slopes_of

pytestmark = pytest.mark.gpu
KS, VS = 0.011, 0.37


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def make(B, H, Hkv, d, ctx, seed, begin=None, spare=2):
    per = [(c + 15) // 16 for c in ctx]
    width = max(1, max(per)) + spare
    k, v, nan = F.pool(sum(per), Hkv, d, seed, 0.02)
    g = torch.Generator().manual_seed(seed + 1)
    perm = torch.randperm(sum(per), generator=g)
    table = torch.full((B, width), nan, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
        if ctx[b] % 16:
            F.poison(k, v, int(table[b, n - 1]), ctx[b] % 16, 16)
        if begin is not None and 0 < begin[b] < ctx[b]:
            table[b, :begin[b] // 16] = nan
            F.poison(k, v, int(table[b, begin[b] // 16]), 0, begin[b] % 16)
    q = (torch.randn(B, H, d, generator=g) * 2).to(torch.bfloat16)
    return q, k, v, table, torch.tensor(ctx, dtype=torch.int32)


def run(lib, x, **kw):
    q, k, v, table, ctx = (t.cuda() for t in x)
    kw = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in kw.items()}
    return lib.paged_attn_decode_fp4(q, k, v, KS, VS, table, ctx, **kw)


def want(x, scale, cap=0.0, slopes=None, begin=None):
    q, k, v, table, ctx = x
    return R.decode(q, F.read(k, False) * KS, F.read(v, True) * VS, table, [int(c) for c in ctx], scale, False, cap, slopes, begin)


@pytest.mark.parametrize("mod", [(0.0, False, 0), (5.0, False, 0), (0.0, True, 100), (30.0, True, 33)],
                         ids=["plain", "cap5", "bias_window", "cap30_bias_window"])
@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=[f"B{s[0]}H{s[1]}kv{s[2]}d{s[3]}" for s in SHAPES])
def test_matches_the_definition(lib, shape, spare, mod):
    B, H, Hkv, d, ctx = shape
    cap, bias, window = mod
    begin = [c - window for c in ctx] if window else None
    x = make(B, H, Hkv, d, ctx, 3, begin, spare)
    sl = slopes_of(H) if bias else None
    kb = None if begin is None else torch.tensor(begin, dtype=torch.int32)
    o = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), float("nan"), device="cuda")
    scale = 2 * d ** -0.5
    run(lib, x, scale=scale, softcap=cap, alibi_slopes=sl, key_begin=kb, out=o, lse=lse)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    R.check(o.cpu(), lse.cpu(), *want(x, scale, cap, sl, begin))


@pytest.mark.parametrize("d", [32, 64, 80, 96, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 16, 17])
def test_every_head_dim_and_group(lib, d, group):
    ctx = [47, 16, 301]
    x = make(3, 2 * group, 2, d, ctx, 4)
    out = run(lib, x)
    R.check(out[0].cpu(), out[1].cpu(), *want(x, d ** -0.5))


@pytest.mark.parametrize("spare", [0, WIDE], ids=["cluster", "workspace"])
def test_unmapped_pages_and_odd_intervals(lib, spare):
    ctx = [200, 300, 64, 500, 5000, 50, -4, 2**31 - 1]
    begin = [200, 2**31 - 1, -5, 250, 10, 50, 0, 4990]  # nothing left, nothing left, all, a page's middle, ...
    x = make(8, 4, 2, 64, [min(max(c, 0), 4992) for c in ctx], 5, spare=spare)
    x[3][0, 1], x[3][3, 20], x[3][2, 0] = -1, 10**6, -7
    x[3][5, :] = x[1].shape[0]  # no page mapped at all
    x[3][4, 312:] = x[3][7, 312:] = -1  # (4992 tokens and no more)
    seen = [min(max(c, 0), 16 * x[3].shape[1]) for c in ctx]
    out = run(lib, (*x[:4], torch.tensor(ctx, dtype=torch.int32)), softcap=10.0, alibi_slopes=slopes_of(4),
              key_begin=torch.tensor(begin, dtype=torch.int32))
    w = want((*x[:4], seen), 64 ** -0.5, 10.0, slopes_of(4), begin)
    # biases of thousands: the score nearest to 0, its sum with the log of the weights and that times ln 2 are each rounded
    # to fp32, by 2^-24 of LSE (here |LSE| up to 8400: 5e-4 each); what is beyond that is held to the bound
    off = (out[1].cpu().double() - w[1]).nan_to_num(0.0)
    most = (3 * 2.0 ** -24 * w[1].abs()).nan_to_num(0.0, posinf=0.0)
    R.check(out[0].cpu(), torch.where(torch.isinf(w[1]), out[1].cpu().double(), w[1] + off - off.clamp(-most, most)), *w)


@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("d", [32, 64, 80, 96, 128])
def test_a_window_alone(lib, d, spare):
    ctx, window = [700, 16, 1, 2049, 33], [100, 16, 5, 1, 2]
    begin = [c - w for c, w in zip(ctx, window)]
    x = make(5, 6, 2, d, ctx, 11, begin, spare)
    out = run(lib, x, key_begin=torch.tensor(begin, dtype=torch.int32))
    R.check(out[0].cpu(), out[1].cpu(), *want(x, d ** -0.5, 0.0, None, begin))


def test_large_batches_of_uneven_lengths(lib):
    # more sequences than a share's search takes in one go, most of them empty or a few tokens long, one of them long
    for B, H, Hkv, d in ((1500, 2, 1, 32), (700, 24, 2, 64)):
        g = torch.Generator().manual_seed(B)
        ctx = (torch.rand(B, generator=g) ** 6 * 60).int().tolist()
        ctx[B // 3] = 5000
        x = make(B, H, Hkv, d, ctx, 12)
        out = run(lib, x)
        R.check(out[0].cpu(), out[1].cpu(), *want(x, d ** -0.5))


def test_huge_and_nan_queries(lib):
    x = list(make(3, 4, 2, 64, [40, 90, 33], 7))
    x[0] = (x[0].float() * 2.0 ** 20).to(torch.bfloat16)
    scale = 2.0 ** -20
    out = run(lib, x, scale=scale, softcap=20.0)
    R.check(out[0].cpu(), out[1].cpu(), *want(x, scale, 20.0))
    y = list(x)
    y[0] = x[0].clone()
    y[0][1, 2, 5] = float("nan")
    bad = run(lib, y, scale=scale, softcap=20.0)
    assert bad[0][1, 2].isnan().all() and bad[1][1, 2].isnan()
    rest = torch.ones(3, 4, dtype=torch.bool)
    rest[1, 2] = False
    assert torch.equal(bad[0].cpu()[rest], out[0].cpu()[rest]) and torch.equal(bad[1].cpu()[rest], out[1].cpu()[rest])


def test_extreme_scales_of_blocks(lib):
    # block scales from the smallest (2^-9) to the largest (448) side by side, of both signs
    x = list(make(2, 8, 2, 128, [100, 37], 8))
    g = torch.Generator().manual_seed(1)
    for p in (x[1], x[2]):
        p[:-1, :, 8 * 128:] = torch.tensor([0x01, 0x7E, 0x38, 0x81, 0x00, 0xB8], dtype=torch.uint8)[
            torch.randint(0, 6, p[:-1, :, 8 * 128:].shape, generator=g)]
    out = run(lib, x, scale=0.01)
    R.check(out[0].cpu(), out[1].cpu(), *[t for t in want([*x[:3], torch.where(x[3] == x[1].shape[0] - 1, -1, x[3]), x[4]], 0.01)])


def test_many_rows_with_few_splits(lib):
    for B in (32, 64):
        ctx = [(b * 97) % 1200 for b in range(B)]
        x = make(B, 8, 8, 32, ctx, 9)
        out = run(lib, x, softcap=20.0)
        R.check(out[0].cpu(), out[1].cpu(), *want(x, 32 ** -0.5, 20.0))


@pytest.mark.parametrize("spare", **FORMS)
def test_other_stream_graph_and_workspace(lib, spare):
    x = make(3, 8, 2, 64, [300, 17, 1500], 8, spare=spare)
    w = run(lib, x, softcap=20.0)
    side = torch.cuda.Stream()
    q, k, v, table, ctx = (t.cuda() for t in x)
    need = lib.paged_attn_decode_fp4_workspace_size(3, 8, 2, 64, table.shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = lib.paged_attn_decode_fp4(q, k, v, KS, VS, table, ctx, softcap=20.0, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    with pytest.raises(lib.AttnError):
        lib.paged_attn_decode_fp4(q, k, v, KS, VS, table, ctx, workspace=ws[:need - 16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = lib.paged_attn_decode_fp4(q, k, v, KS, VS, table, ctx, softcap=20.0)
    graph.replay()
    ctx.copy_(torch.tensor([100, 16, 1491], dtype=torch.int32))  # lengths are read at each replay
    graph.replay()
    w = lib.paged_attn_decode_fp4(q, k, v, KS, VS, table, ctx, softcap=20.0)
    assert torch.equal(cap[0], w[0]) and torch.equal(cap[1], w[1])


@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_sixteen_million_tokens(lib, cap):
    """A context of 2^20 pages, the same 64 over and over: the result is theirs, with ln(2^14) more in LSE.

    A lane adds at most 4 weights of each of its warp's pages (2^21 rows' pages over 2432 warps: 863) to its sum, a chain of
    3452 roundings of 2^-24: 2.1e-4 relative, and so in LSE.  O, of the largest value: the weights' rounding to f16 (2^-11, here
    2^-10) and 863 roundings of an accumulator, a few 2^-24 each (2^-12); of O: the sum's error and the rounding to bf16."""
    x = make(1, 4, 2, 64, [1024], 21, spare=0)
    o, lse = want(x, 0.125, cap)[:2]
    table = x[3].repeat(1, 1 << 14)
    ctx = torch.tensor([1 << 24], dtype=torch.int32)
    got = run(lib, (x[0], x[1], x[2], table, ctx), scale=0.125, softcap=cap)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    more = torch.log(torch.tensor(2.0 ** 14, dtype=torch.float64))
    assert (got[1].cpu().double() - (lse + more)).abs().max() <= 3e-4
    top = (F.read(x[2], True) * VS)[x[3][0].long()].abs().max()
    bound = (2.0 ** -8 + 2.0 ** -12) * o.abs() + (2.0 ** -10 + 2.0 ** -12) * top
    assert ((got[0].cpu().double() - o).abs() <= bound).all()
    # the last 1000 tokens alone, by a window
    short = run(lib, (x[0], x[1], x[2], table, ctx), scale=0.125, softcap=cap, key_begin=torch.tensor([(1 << 24) - 1000], dtype=torch.int32))
    begin = [24]
    R.check(short[0].cpu(), short[1].cpu(), *want(x, 0.125, cap, None, begin))
