"""Rotation by positions with several axes, and its gradient, against the definition in 64 bits; and the append by such
positions against the plain append.

A rotated value is x cos - y sin in fp32, off by at most 2^-22 (|x| + |y|), rounded once to bf16 (2^-8 of itself)."""
import pytest
import torch

from test_gpu_append_rope import angles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def rnd(g, *s):
    return torch.randn(*s, generator=g).to(torch.bfloat16)


def want(x, pos, pair, cs, inter, back):
    """x [B, heads, N, d] in float64 turned, and the slack of fp32; zeros for tokens outside the table."""
    r = cs.shape[1]
    i = torch.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    row = pos[torch.tensor(list(pair))].expand(-1, x.shape[0], -1).permute(1, 2, 0)  # [B, N, pairs]
    ok = ((pos >= 0) & (pos < cs.shape[0])).all(0).expand(x.shape[0], -1)
    row = row.clamp(0, cs.shape[0] - 1)
    c, s = cs[row, i].double()[:, None], cs[row, r // 2 + i].double()[:, None] * (-1 if back else 1)
    out, slack = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    xa, xb = out[..., a].clone(), out[..., b].clone()
    out[..., a], out[..., b] = xa * c - xb * s, xb * c + xa * s
    slack[..., a] = slack[..., b] = 2.0 ** -22 * (xa.abs() + xb.abs())
    return out * ok[:, None, :, None], slack


CASES = [  # B, H, Hkv, N, d, rope, axes
    (1, 1, 1, 1, 32, 32, 1), (3, 12, 12, 5, 64, 64, 3), (2, 7, 1, 18, 80, 80, 2), (2, 4, 2, 37, 96, 48, 4), (3, 32, 8, 4, 128, 128, 3),
    (2, 6, 2, 131, 128, 64, 2), (1, 2, 0, 301, 32, 16, 3),
]


@pytest.mark.parametrize("back", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("shared", [False, True], ids=["each", "shared"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}H{c[1]}kv{c[2]}N{c[3]}d{c[4]}r{c[5]}a{c[6]}" for c in CASES])
def test_matches_the_definition(lib, case, shared, inter, back):
    B, H, Hkv, N, d, r, A = case
    g = torch.Generator().manual_seed(5)
    qkv = rnd(g, B, N, H + 2 * Hkv, d).cuda().transpose(1, 2)
    x = [qkv[:, :H], qkv[:, H:H + Hkv] if Hkv else None]
    pos = torch.randint(0, 50, (A, 1 if shared else B, N), generator=g)
    if N > 3:
        pos[0, 0, 2], pos[A - 1, 0, 3] = -1, 50  # outside the table
    pair, cs = bytes(torch.randint(0, A, (r // 2,), generator=g).tolist()), angles(50, r) * 1.25  # with a factor on c and s
    f = lib.attn_rope_axes_bwd if back else lib.attn_rope_axes
    arg = (cs.cuda(), pos.int().cuda(), pair, inter)
    out = f(*x, *arg)
    assert (out[1] is None) == (Hkv == 0)
    dense = [None if t is None else t.clone(memory_format=torch.contiguous_format) for t in x]
    into = torch.full((B, N, H + 2 * Hkv, d), 3.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    views = [into[:, :H], into[:, H:H + Hkv] if Hkv else None]
    r2 = f(*dense, *arg, q_out=views[0], k_out=views[1])
    assert r2[0] is views[0] and r2[1] is views[1] and (into[:, H + Hkv:] == 3).all()
    for t, o, v, y in zip(x, out, views, dense):
        if t is None:
            continue
        w, slack = want(t.cpu(), pos, pair, cs, inter, back)
        assert ((o.cpu().double() - w).abs() <= 2.0 ** -8 * w.abs() + slack).all()
        assert torch.equal(o, v)
    same = f(*dense, *arg, q_out=dense[0], k_out=dense[1])  # in place
    assert all(a is None or torch.equal(a, b) for a, b in zip(same, out))
    f(*x, *arg, q_out=x[0], k_out=x[1])  # the views in place
    assert torch.equal(x[0], out[0]) and (x[1] is None or torch.equal(x[1], out[1]))


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
def test_gradient_against_differences(lib, inter):
    """sum(w * rope(x)) is linear in x: its difference along e is the gradient's product with e, up to the roundings to bf16
    of the outputs (2^-8 of each, summed with the weights w) and of the gradient (2^-8 of each, with e)."""
    g = torch.Generator().manual_seed(6)
    x, e, w = (rnd(g, 2, 3, 9, 64).cuda() for _ in range(3))
    arg = (angles(30, 48).cuda(), torch.randint(0, 30, (3, 2, 9), generator=g).int().cuda(), bytes(i % 3 for i in range(24)), inter)
    grad = lib.attn_rope_axes_bwd(w, None, *arg)[0].double()
    hi, lo = ((x.float() + s * e.float()).to(torch.bfloat16) for s in (8, -8))
    y1, y0 = (lib.attn_rope_axes(t, None, *arg)[0].double() for t in (hi, lo))
    diff, moved = (w.double() * (y1 - y0)).sum(), hi.double() - lo.double()
    tol = 2.0 ** -8 * ((w.double() * y1).abs().sum() + (w.double() * y0).abs().sum() + (grad * moved).abs().sum()) * 1.01
    assert (diff - (grad * moved).sum()).abs() <= tol and tol < 0.05 * (w.double() * y1).abs().sum()


def test_one_axis_is_the_plain_append_and_text_too(lib):
    """Equal positions on every axis are the plain rotation, bit for bit, in every cache's append."""
    B, H, Hkv, N, d, r = 3, 4, 2, 21, 64, 64
    g = torch.Generator().manual_seed(7)
    qkv = rnd(g, B, N, H + 2 * Hkv, d).cuda().transpose(1, 2)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    start = torch.tensor([0, 5, 30], dtype=torch.int32)
    pos = (start[:, None] + torch.arange(N)).int().expand(3, B, N).contiguous().cuda()
    table, cs = torch.arange(B * 4, dtype=torch.int32).view(B, 4).cuda(), angles(64, r).cuda()
    new = torch.tensor([21, 0, 20], dtype=torch.int32).cuda()
    start = start.cuda()
    for inter in (False, True):
        for name, shape, dtype, scales in (("rope", (16, d), torch.bfloat16, ()), ("rope_fp8", (16, d), torch.uint8, (0.02, 0.013)),
                                           ("fp4", (9 * d,), torch.uint8, (0.02, 0.013))):
            pools = [[torch.zeros(B * 4, Hkv, *shape, dtype=dtype, device="cuda") for _ in range(2)] for _ in range(2)]
            o = [torch.zeros(B, H, N, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            for way, (p, out) in enumerate(zip(pools, o)):
                kw = dict(interleaved=inter, new_lens=new, q_out=out)
                pair = [i % 3 for i in range(r // 2)]
                if name == "fp4":
                    more = dict(positions=pos, pair_axis=bytes(pair)) if way else {}
                    lib.paged_kv_append_fp4(q, k, v, *p, *scales, table, start, cos_sin=cs, **more, **kw)
                elif way:
                    f = lib.paged_kv_append_rope_axes_fp8 if scales else lib.paged_kv_append_rope_axes
                    f(q, k, v, *p, *scales, cs, pos, pair, table, start, **kw)
                else:
                    f = lib.paged_kv_append_rope_fp8 if scales else lib.paged_kv_append_rope
                    f(q, k, v, *p, *scales, cs, table, start, **kw)
            assert torch.equal(*o) and all(torch.equal(a, b) for a, b in zip(*pools)), (name, inter)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("case", CASES[:-1], ids=[f"d{c[4]}r{c[5]}a{c[6]}N{c[3]}" for c in CASES[:-1]])
def test_append_is_the_rotation_and_the_copy(lib, case, inter, fp8):
    B, H, Hkv, N, d, r, A = case
    g = torch.Generator().manual_seed(8)
    qkv = rnd(g, B, N, H + 2 * Hkv, d).cuda().transpose(1, 2)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    pos = torch.randint(0, 50, (A, B, N), generator=g)
    bad = torch.zeros(B, N, dtype=torch.bool)
    if N > 3:
        pos[A - 1, 0, 3], bad[0, 3] = 50, True
    pair, cs = bytes(torch.randint(0, A, (r // 2,), generator=g).tolist()), angles(50, r)
    start = torch.tensor([1000 * b + 7 for b in range(B)], dtype=torch.int32)  # the place is not the position
    W = (int(start.max()) + N) // 16 + 2
    table = torch.full((B, W), -1, dtype=torch.int32)
    used = torch.zeros(B, W, dtype=torch.bool)
    for b in range(B):
        used[b, int(start[b]) // 16:(int(start[b]) + N - 1) // 16 + 1] = True
    table[used] = torch.randperm(int(used.sum()), generator=g).int()
    P = int(used.sum())
    pools = [torch.zeros(P, Hkv, 16, d, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2)]
    q_out = torch.full((B, H, N, d), 7.0, dtype=torch.bfloat16, device="cuda")
    scales = (0.02, 0.013) if fp8 else ()
    f = lib.paged_kv_append_rope_axes_fp8 if fp8 else lib.paged_kv_append_rope_axes
    f(q, k, v, *pools, *scales, cs.cuda(), pos.int().cuda(), pair, table.cuda(), start.cuda(), interleaved=inter, q_out=q_out)
    turned = lib.attn_rope_axes(q, k, cs.cuda(), pos.int().cuda(), pair, inter)
    assert torch.equal(q_out[~bad[:, None].expand(B, H, N)], turned[0][~bad[:, None].expand(B, H, N)])
    assert (q_out.cpu()[bad[:, None].expand(B, H, N)] == 7).all()
    wk, slack = want(k.cpu(), pos, pair, cs, inter, False)
    for b in range(B):
        for t in range(N):
            at = int(start[b]) + t
            page, slot = int(table[b, at // 16]), at % 16
            got = [p[page, :, slot].cpu() for p in pools]
            if bad[b, t]:
                assert all(int(x.view(torch.uint8).max()) == 0 for x in got)
            elif fp8:
                u = (wk[b, :, t] / 0.02).clamp(-448, 448)
                err = (got[0].view(torch.float8_e4m3fn).double() - u).abs()
                assert (err <= torch.maximum(2.0 ** -4 * u.abs(), torch.full_like(u, 2.0 ** -10)) + (slack[b, :, t] + 2.0 ** -22 * wk[b, :, t].abs()) / 0.02).all()
            else:
                assert torch.equal(got[0], turned[1][b, :, t].cpu()) and torch.equal(got[1], v[b, :, t].cpu())


def test_other_stream_graph_and_long_views(lib):
    g = torch.Generator().manual_seed(9)
    q, k = rnd(g, 2, 4, 33, 64).cuda(), rnd(g, 2, 2, 33, 64).cuda()
    pos, cs, pair = torch.randint(0, 40, (3, 2, 33), generator=g).int().cuda(), angles(40, 64).cuda(), bytes([0] * 8 + [1] * 12 + [2] * 12)
    w = lib.attn_rope_axes(q, k, cs, pos, pair)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = lib.attn_rope_axes(q, k, cs, pos, pair, stream=side)
    side.synchronize()
    assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = lib.attn_rope_axes(q, k, cs, pos, pair)
    pos.copy_(pos.flip(2))
    graph.replay()
    w = lib.attn_rope_axes(q, k, cs, pos, pair)
    assert torch.equal(cap[0], w[0]) and torch.equal(cap[1], w[1])
    # heads 2^30 elements apart: the last rows lie past every 32-bit offset
    big = torch.empty(3 << 30, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((1, 3, 33, 64), (0, 1 << 30, 64, 1))
    far.copy_(q[:1, :3])
    a, b = lib.attn_rope_axes(far, None, cs, pos[:, :1].contiguous(), pair)[0], lib.attn_rope_axes(q[:1, :3].contiguous(), None, cs, pos[:, :1].contiguous(), pair)[0]
    assert torch.equal(a, b)
    lib.attn_rope_axes(q[:1, :3].contiguous(), None, cs, pos[:, :1].contiguous(), pair, q_out=far)
    assert torch.equal(far, b)
