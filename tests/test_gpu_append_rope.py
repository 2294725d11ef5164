"""Append with rotation against its definition in 64 bits.

Tolerances, from the roundings that happen: a rotated value is x cos - y sin in fp32, off by at most
2^-22 (|x| + |y|), and is then rounded once, by at most 2^-8 of itself to bf16, or by 2^-4 of itself
(2^-10 below the normal range) to e4m3 after the factor 1 / scale (off by 2^-23)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
PS = 16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def angles(max_pos, r):
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate64(x, cs, inter):
    """x [heads, n, d] float64, cs [n, r] float64."""
    r = cs.shape[1]
    x, c, s = x.clone(), cs[:, :r // 2], cs[:, r // 2:]
    i = torch.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    xa, xb = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    slack = torch.zeros_like(x)
    slack[..., a] = slack[..., b] = 2.0 ** -22 * (xa.abs() + xb.abs())
    return x, slack


def values(t, fp8):
    return t.view(torch.float8_e4m3fn).double() if fp8 else t.double()


def make(B, H, Hkv, N, d, r, fp8, start, max_pages, max_pos, seed, fused=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    if fused:  # [B, N, heads, d] projections, as views
        qkv = rnd(B, N, H + 2 * Hkv, d).cuda().transpose(1, 2)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        q, k, v = rnd(B, H, N, d).cuda(), rnd(B, Hkv, N, d).cuda(), rnd(B, Hkv, N, d).cuda()
    num_pages = B * max_pages + 1
    table = torch.randperm(num_pages - 1, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32).cuda()
    pool = [rnd(num_pages, Hkv, PS, d).cuda() for _ in range(2)]
    if fp8:
        pool = [p.float().to(torch.float8_e4m3fn).view(torch.uint8) for p in pool]
    return dict(q=q, k=k, v=v, kp=pool[0], vp=pool[1], table=table, cs=angles(max_pos, r).cuda(),
                start=torch.tensor(start, dtype=torch.int32).cuda())


def check(x, before, q_out, q_before, inter, fp8, scales, new=None):
    """Every slot and query row: the written ones within tolerance, the others bit for bit as before."""
    q, k, v = x["q"].cpu().double(), x["k"].cpu().double(), x["v"].cpu().double()
    B, H, N, d = q.shape
    cs, table = x["cs"].cpu().double(), x["table"].cpu()
    got = [values(p.cpu(), fp8) for p in (x["kp"], x["vp"])]
    touched = torch.zeros(got[0].shape[0], PS, dtype=torch.bool)
    qo = q_out.cpu()
    qt = torch.zeros(B, N, dtype=torch.bool)
    inv = [1.0 / s for s in scales]
    half, least = (2.0 ** -4, 2.0 ** -10) if fp8 else (2.0 ** -8, 0.0)
    for b in range(B):
        n = N if new is None else min(max(new[b], 0), N)
        start = max(int(x["start"][b]), 0)
        n = max(0, min(n, cs.shape[0] - start))  # tokens past the rotation table are padding
        if n == 0:
            continue
        rows = cs[start:start + n]
        want, slack = rotate64(q[b, :, :n], rows, inter)
        assert ((qo[b, :, :n].double() - want).abs() <= 2.0 ** -8 * want.abs() + slack).all()
        qt[b, :n] = True
        kr, ks = rotate64(k[b, :, :n], rows, inter)
        for t in range(n):
            pos = start + t
            if pos // PS >= table.shape[1]:
                continue
            page = int(table[b, pos // PS])
            if page < 0 or page >= got[0].shape[0]:
                continue
            touched[page, pos % PS] = True
            for have, w, sl, i in ((got[0], kr[:, t], ks[:, t], 0), (got[1], v[b, :, t], 0 * ks[:, t], 1)):
                w = (w * inv[i]).clamp(-448, 448) if fp8 else w
                tol = torch.maximum(half * w.abs(), torch.full_like(w, least)) + sl * inv[i] + 2.0 ** -22 * w.abs()
                err = (have[page, :, pos % PS] - w).abs()
                assert (err <= (tol if i == 0 or fp8 else 0 * tol)).all(), (b, t, i, float(err.max()))
    for p, old in zip((x["kp"], x["vp"]), before):
        keep = ~touched[:, None, :, None].expand(p.shape)
        assert torch.equal(p.cpu()[keep], old.cpu()[keep])
    keep = ~qt[:, None, :, None].expand(qo.shape)
    assert torch.equal(qo[keep].view(torch.int16), q_before.cpu()[keep].view(torch.int16))


def call(lib, x, fp8, scales, inter, **kw):
    if fp8:
        return lib.paged_kv_append_rope_fp8(x["q"], x["k"], x["v"], x["kp"], x["vp"], *scales, x["cs"], x["table"],
                                            x["start"], interleaved=inter, **kw)
    return lib.paged_kv_append_rope(x["q"], x["k"], x["v"], x["kp"], x["vp"], x["cs"], x["table"], x["start"],
                                    interleaved=inter, **kw)


CASES = [  # B, H, Hkv, N, d, rope, start
    (1, 1, 1, 1, 32, 32, [0]),
    (3, 12, 12, 1, 64, 64, [0, 15, 600]),
    (2, 7, 1, 5, 80, 80, [14, 31]),
    (2, 4, 2, 37, 96, 48, [0, 201]),
    (3, 32, 8, 1, 128, 64, [17, 0, 320]),
    (2, 6, 2, 130, 128, 128, [3, 250]),
    (1, 2, 2, 301, 32, 16, [9]),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}H{c[1]}kv{c[2]}N{c[3]}d{c[4]}r{c[5]}" for c in CASES])
def test_matches_the_definition(lib, case, inter, fp8):
    B, H, Hkv, N, d, r, start = case
    scales = (0.02, 0.013) if fp8 else (1.0, 1.0)
    for fused in (True, False):
        x = make(B, H, Hkv, N, d, r, fp8, start, (max(start) + N + 15) // 16 + 1, max(start) + N, 5, fused)
        before = [x["kp"].clone(), x["vp"].clone()]
        q_out = torch.full((B, H, N, d), 7.0, dtype=torch.bfloat16, device="cuda")
        old = q_out.clone()
        assert call(lib, x, fp8, scales, inter, q_out=q_out) is q_out
        torch.cuda.synchronize()
        check(x, before, q_out, old, inter, fp8, scales)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_padding_unmapped_pages_and_ends(lib, fp8):
    scales = (0.02, 0.013) if fp8 else (1.0, 1.0)
    # sequence 0: nothing new; 1: part; 2: past the page table's capacity; 3: negative start; 4: more than Nnew
    start, new = [5, 40, 60, -3, 0], [0, 9, 21, 21, 1000]
    x = make(5, 4, 2, 21, 64, 32, fp8, start, 4, 70, 6)
    x["table"][1, 2] = -1                   # unmapped
    x["table"][3, 0] = x["kp"].shape[0]     # outside the pool
    before = [x["kp"].clone(), x["vp"].clone()]
    q_out = torch.full((5, 4, 21, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    old = q_out.clone()
    call(lib, x, fp8, scales, False, q_out=q_out, new_lens=torch.tensor(new, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    check(x, before, q_out, old, False, fp8, scales, new)


def test_start_at_the_largest_int(lib):
    x = make(2, 2, 2, 3, 64, 64, False, [2**31 - 1, 1], 2, 8, 7)
    before = [x["kp"].clone(), x["vp"].clone()]
    q_out = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    old = q_out.clone()
    call(lib, x, False, (1, 1), False, q_out=q_out)
    torch.cuda.synchronize()
    check(x, before, q_out, old, False, False, (1.0, 1.0))


@pytest.mark.parametrize("inter", [False, True])
def test_query_in_place_and_keys_only(lib, inter):
    x = make(2, 4, 2, 19, 128, 96, False, [3, 30], 4, 64, 8, fused=False)
    y = make(2, 4, 2, 19, 128, 96, False, [3, 30], 4, 64, 8, fused=False)
    out = call(lib, x, False, (1, 1), inter)
    y["q_same"] = y["q"]
    assert call(lib, y, False, (1, 1), inter, q_out=y["q"]) is y["q"]
    assert torch.equal(out, y["q"]) and torch.equal(x["kp"], y["kp"]) and torch.equal(x["vp"], y["vp"])
    z = make(2, 4, 2, 19, 128, 96, False, [3, 30], 4, 64, 8, fused=False)
    z["q"] = None
    assert call(lib, z, False, (1, 1), inter) is None
    assert torch.equal(x["kp"], z["kp"]) and torch.equal(x["vp"], z["vp"])


def test_other_stream_and_captured_graph(lib):
    x = make(4, 8, 2, 1, 128, 128, False, [0, 5, 15, 33], 4, 64, 9)
    ref = make(4, 8, 2, 1, 128, 128, False, [0, 5, 15, 33], 4, 64, 9)
    want = call(lib, ref, False, (1, 1), False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(lib, x, False, (1, 1), False, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(x["kp"], ref["kp"])
    # one decode step after the other from one captured call: the position advances on the device
    y = make(4, 8, 2, 1, 128, 128, False, [0, 5, 15, 33], 4, 64, 10)
    z = make(4, 8, 2, 1, 128, 128, False, [0, 5, 15, 33], 4, 64, 10)
    q_out = torch.zeros(4, 8, 1, 128, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(lib, y, False, (1, 1), False, q_out=q_out)
    for step in range(3):
        graph.replay()
        want = call(lib, z, False, (1, 1), False)
        torch.cuda.synchronize()
        assert torch.equal(q_out, want) and torch.equal(y["kp"], z["kp"]) and torch.equal(y["vp"], z["vp"])
        y["start"].add_(1)
        z["start"].add_(1)


def test_pool_past_32_bit_offsets(lib):
    # a pool of more than 2^31 elements: the last pages lie past every 32-bit offset
    Hkv, d = 8, 128
    pages = (1 << 31) // (Hkv * PS * d) + 64
    kp = torch.zeros(pages, Hkv, PS, d, dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    g = torch.Generator().manual_seed(11)
    k = torch.randn(1, Hkv, 20, d, generator=g).to(torch.bfloat16).cuda()
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    start = torch.tensor([7], dtype=torch.int32, device="cuda")
    cs = angles(32, d).cuda()
    lib.paged_kv_append_rope_fp8(None, k, k, kp, vp, 0.02, 0.02, cs, table, start)
    small = torch.zeros(4, Hkv, PS, d, dtype=torch.uint8, device="cuda")
    svp = torch.zeros_like(small)
    lib.paged_kv_append_rope_fp8(None, k, k, small, svp, 0.02, 0.02, cs, torch.tensor([[3, 1]], dtype=torch.int32).cuda(), start)
    assert torch.equal(kp[-4:], small) and torch.equal(vp[-4:], svp)
    assert int(kp[:-4].max()) == 0 and int(vp[:-4].max()) == 0


def test_append_then_decode(lib):
    """The append as it is used: a chunk and then single tokens go in, and the decode reads them."""
    B, H, Hkv, d, n = 2, 4, 2, 64, 33
    x = make(B, H, Hkv, n, d, d, False, [0, 0], 4, 64, 12)
    y = make(B, H, Hkv, n, d, d, False, [0, 0], 4, 64, 12)
    whole = call(lib, x, False, (1, 1), False)
    start = y["start"].clone()
    lib.paged_kv_append_rope(y["q"][:, :, :20], y["k"][:, :, :20], y["v"][:, :, :20], y["kp"], y["vp"], y["cs"], y["table"], start)
    for t in range(20, n):
        start.fill_(t)
        last = lib.paged_kv_append_rope(y["q"][:, :, t:t + 1], y["k"][:, :, t:t + 1], y["v"][:, :, t:t + 1], y["kp"], y["vp"],
                                        y["cs"], y["table"], start)
    assert torch.equal(x["kp"], y["kp"]) and torch.equal(x["vp"], y["vp"]) and torch.equal(last, whole[:, :, n - 1:])
    ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
    o, _ = lib.paged_attn_decode_gqa(last.view(B, H, d), y["kp"], y["vp"], y["table"], ctx)
    cs = x["cs"].cpu().double()[:n]
    for b in range(B):
        for h in range(H):
            kr, _ = rotate64(x["k"][b, h // 2].cpu().double()[None], cs, False)
            qr, _ = rotate64(x["q"][b, h].cpu().double()[None], cs, False)
            p = torch.softmax(kr[0] @ qr[0, -1] * d ** -0.5, 0)
            want = p @ x["v"][b, h // 2].cpu().double()
            # scores move by at most the 2^-8 of each rotated factor: |s| <= about 4 standard deviations
            # of unit scores over rows of norm sqrt(d), so weights by about 2 * 2^-8 * 4 and o by that of |v| <= 4
            assert (o[b, h].cpu().double() - want).abs().max() <= 2 * 2.0 ** -8 * 4 * 4 + 2.0 ** -8 * 4
    assert lib.attn_check_device_status() == 0
