"""Attention with modified scores (tanh cap, distance bias, key intervals) against its definition in
64 bits.

Tolerances.  O = sum_j w_j v_j / l: every weight is rounded once to bf16 (off by at most 2^-8 of itself),
l sums them unrounded, O is rounded once (2^-8 of itself).  A score is a sum of d <= 128 exact products in
fp32, off by at most 128 * 2^-23 of scale * sum |q k| (about 14 for the largest inputs here, so 2e-4), which
moves a weight and l by that much each.  So, with W|v| = sum_j w_j |v_j| of the definition,
    |O - O_64| <= (2^-8 + 4e-4) W|v| + 2^-8 |O|   (the cross terms: 1 % more),
element by element.  The mean bound (the other parity tests') is an average over random signs.  LSE: the
scores' error adds up like sqrt(d) and not d over random signs: 1e-4."""
import pytest
import torch

from scoremod_ref import backward, documents, forward, prefix

pytestmark = pytest.mark.gpu
O_MEAN, LSE_MAX = 1e-3, 1e-4


def o_bound(w, v, o):
    wv = w @ v.double().nan_to_num(0.0, 0.0, 0.0).abs().repeat_interleave(w.shape[1] // v.shape[1], 1)
    return 1.01 * ((2.0 ** -8 + 4e-4) * wv + 2.0 ** -8 * o.abs()) + 1e-30


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def rand(seed, *shape, by=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * by).to(torch.bfloat16)


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])


def cuda(t):
    return None if t is None else t.cuda()


def masks(kind, B, Nq, Nkv):
    kw = dict(causal=False, key_begin=None, key_end=None, kv_lens=None)
    if kind == "causal":
        kw["causal"] = True
    elif kind == "docs":
        kw["causal"] = True
        kw["key_begin"], kw["key_end"] = documents(B, Nq, Nkv, [1, 70, 300, 16, 129])
    elif kind == "docs_both_ways":
        kw["key_begin"], kw["key_end"] = documents(B, Nq, Nkv, [128, 1, 55, 200])
    elif kind == "prefix_padded":
        kw["key_end"] = prefix(B, Nq, Nkv, [0, Nkv // 3, Nkv])
        kw["kv_lens"] = torch.tensor([Nkv - (b * 37) % max(1, Nkv) for b in range(B)], dtype=torch.int32)
    elif kind == "window":
        p = torch.arange(Nq) + (Nkv - Nq)
        kw["causal"] = True
        kw["key_begin"] = (p - 49).expand(B, Nq).contiguous().to(torch.int32)
    elif kind == "empty_rows":  # documents past the keys, intervals turned round, keys gone
        kw["key_begin"], kw["key_end"] = documents(B, Nq, Nkv, [90, 40])
        kw["kv_lens"] = torch.tensor([Nkv // 2, 0, 1, Nkv][:B] + [Nkv] * (B - 4), dtype=torch.int32)
        kw["key_end"][:, ::5] = -7
        kw["key_end"][:, 3::11] = -2**31
        kw["key_begin"][:, 1::11] = -2**31
        kw["key_begin"][:, ::7] = 2**31 - 1
        kw["key_end"][:, 4::13] = 2**31 - 1
    return kw


MASKS = ["none", "causal", "docs", "docs_both_ways", "prefix_padded", "window", "empty_rows"]
SIZES = [  # B, H, Hkv, Nq, Nkv, d
    (2, 2, 2, 1, 1, 32), (1, 3, 1, 65, 64, 64), (2, 4, 2, 300, 300, 80), (1, 2, 1, 129, 517, 96), (3, 2, 2, 257, 256, 128),
    (1, 4, 4, 700, 700, 64), (1, 4, 2, 640, 1000, 128),
]
MODS = [(0.0, False), (5.0, False), (0.0, True), (30.0, True)]


@pytest.mark.parametrize("mod", MODS, ids=["plain", "cap5", "bias", "cap30_bias"])
@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_forward(lib, size, kind, mod):
    B, H, Hkv, Nq, Nkv, d = size
    q, k, v = rand(1, B, H, Nq, d, by=2.0), rand(2, B, Hkv, Nkv, d), rand(3, B, Hkv, Nkv, d)
    cap, bias = mod
    m = masks(kind, B, Nq, Nkv)
    sl = slopes_of(H) if bias else None
    if m["kv_lens"] is not None:  # what lies past the keys may be anything
        for b in range(B):
            n = int(m["kv_lens"][b])
            k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")
    scale = d ** -0.5
    o = torch.full((B, H, Nq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, Nq), float("nan"), device="cuda")
    lib.attn_fwd_scoremod(q.cuda(), k.cuda(), v.cuda(), m["causal"], scale, softcap=cap, alibi_slopes=cuda(sl),
                          key_begin=cuda(m["key_begin"]), key_end=cuda(m["key_end"]), kv_lens=cuda(m["kv_lens"]),
                          out=o, lse=lse)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    want, wl, w, _ = forward(q, k, v, m["causal"], scale, cap, sl, m["key_begin"], m["key_end"], m["kv_lens"])
    err = (o.cpu().double() - want).abs()
    assert torch.isfinite(o).all() and err.mean() <= O_MEAN, float(err.mean())
    assert (err <= o_bound(w, v, want)).all(), float((err / o_bound(w, v, want)).max())
    got = lse.cpu().double()
    assert torch.equal(torch.isneginf(got), torch.isneginf(wl))
    assert (got - wl).nan_to_num(0.0).abs().max() <= LSE_MAX
    empty = torch.isneginf(wl)
    assert (o.cpu()[empty] == 0).all()


def test_plain_call_equals_the_plain_entry_point(lib):
    q, k, v = rand(4, 2, 4, 500, 128).cuda(), rand(5, 2, 2, 500, 128).cuda(), rand(6, 2, 2, 500, 128).cuda()
    for causal in (False, True):
        a = lib.attn_fwd_gqa(q, k, v, causal)
        b = lib.attn_fwd_scoremod(q, k, v, causal)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_large_scores_meet_the_cap(lib):
    # raw scores far beyond the cap: tanh saturates on both sides and the exponential form of tanh runs
    q, k, v = rand(7, 1, 2, 200, 64, by=30.0), rand(8, 1, 2, 200, 64, by=3.0), rand(9, 1, 2, 200, 64)
    for cap in (1.0, 10.0, 50.0):
        o, lse = lib.attn_fwd_scoremod(q.cuda(), k.cuda(), v.cuda(), False, softcap=cap)
        want, wl, w, _ = forward(q, k, v, False, 64 ** -0.5, cap)
        assert (lse.cpu().double() - wl).abs().max() <= 2e-6 * cap + LSE_MAX
        # raw scores reach 30 * 3 * 4 sqrt(d) / sqrt(d) = 400: off by 128 * 2^-23 * scale * sum |q k| <= 9e-3
        # before the cap, whose slope 1 - tanh^2 only shrinks that; all weights move by twice it at most
        assert ((o.cpu().double() - want).abs() <= o_bound(w, v, want) + 1.8e-2 * (w @ v.double().abs())).all()


@pytest.mark.parametrize("cap, scale", [(1e-3, 0.1), (1e-6, 1e-3), (1e6, 0.1), (1e20, 0.1), (1e-20, 0.1), (30.0, 1e-20),
                                        (1e-12, 1e-12), (2.0 ** 100, 0.1)])
def test_extreme_caps(lib, cap, scale):
    q, k, v = rand(13, 1, 2, 150, 64), rand(14, 1, 2, 150, 64), rand(15, 1, 2, 150, 64)
    q[0, 0, 3] = 0  # scores of exactly zero
    q, k, v, g = q.cuda(), k.cuda(), v.cuda(), rand(16, 1, 2, 150, 64).cuda()
    o, lse = lib.attn_fwd_scoremod(q, k, v, True, scale, softcap=cap)
    want, wl, w, t = forward(q, k, v, True, scale, cap)
    assert (lse.cpu().double() - wl).abs().max() <= LSE_MAX
    assert ((o.cpu().double() - want).abs() <= o_bound(w, v.cpu(), want)).all()
    got = lib.attn_bwd_scoremod(q, k, v, o, lse, g, True, scale, softcap=cap)
    ref = backward(q, k, v, g, True, scale, cap)
    # 1 - t^2 where tanh saturates: t is off by at most 2^-22, so the factor by 2^-21
    slack = scale * 2.0 ** -21 * 64
    for x, y, tol in zip(got, ref, grad_bounds(q.cpu(), k.cpu(), v.cpu(), g.cpu(), want, w, t, scale, ref)):
        assert torch.isfinite(x).all()
        assert ((x.cpu().double() - y).abs() <= tol + slack * 150).all()


def test_other_stream_and_captured_graph(lib):
    q, k, v = rand(10, 1, 4, 300, 64).cuda(), rand(11, 1, 4, 300, 64).cuda(), rand(12, 1, 4, 300, 64).cuda()
    kb, ke = (t.cuda() for t in documents(1, 300, 300, [77, 130]))
    want = lib.attn_fwd_scoremod(q, k, v, True, softcap=20.0, key_begin=kb, key_end=ke)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = lib.attn_fwd_scoremod(q, k, v, True, softcap=20.0, key_begin=kb, key_end=ke, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = lib.attn_fwd_scoremod(q, k, v, True, softcap=20.0, key_begin=kb, key_end=ke)
    kb.zero_()
    ke.fill_(300)  # the intervals are read on the device at each replay
    graph.replay()
    want = lib.attn_fwd_scoremod(q, k, v, True, softcap=20.0)
    torch.cuda.synchronize()
    assert torch.equal(cap[0], want[0])


# Gradients.  P and dS are rounded once to bf16 (2^-8 of each) before the products that sum them in fp32, and
# each gradient is rounded once.  D = dO . O is taken from the bf16 O (2^-8 of each O), which moves dP - D by
# at most 2^-8 |dO| . |O|; the scores' error of 2e-4 moves P by 2e-4 of itself.  Element by element, with the
# sums over absolute values of the definition in 64 bits:
#   dV: (2^-8 + 4e-4) P^T |dO|,   dQ, dK: scale (((2^-8 + 4e-4) |dS| + 2^-8 P (|dO| . |O|)) g + 4e-4 |dP - D| P)
#   summed against |K|, |Q| (g = 1 - t^2), each plus 2^-8 of the gradient, 2 % for the cross terms.
def grad_bounds(q, k, v, dout, o64, w, t, scale, grads):
    B, H, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    rep = H // Hkv
    k64, v64 = (x.double().nan_to_num(0.0, 0.0, 0.0).repeat_interleave(rep, 1) for x in (k, v))
    g = dout.double()
    dp = g @ v64.transpose(2, 3) - (g * o64).sum(-1, keepdim=True)
    fac = torch.ones_like(w) if t is None else 1 - t * t
    ds = w * dp.abs() * fac
    slack = w * (g.abs() * o64.abs()).sum(-1, keepdim=True) * fac
    m = scale * ((2.0 ** -8 + 8e-4) * ds + 2.0 ** -8 * slack)
    fold = lambda x: x.view(B, Hkv, rep, Nkv, d).sum(2)  # noqa: E731
    out = (m @ k64.abs(), fold(m.transpose(2, 3) @ q.double().abs()),
           fold((2.0 ** -8 + 4e-4) * (w.transpose(2, 3) @ g.abs())))
    return [1.02 * (b + 2.0 ** -8 * x.abs()) + 1e-9 for b, x in zip(out, grads)]


BWD_SIZES = [(2, 2, 2, 1, 1, 32), (1, 3, 1, 65, 64, 64), (2, 4, 2, 300, 300, 80), (1, 2, 1, 129, 517, 96),
             (3, 2, 2, 257, 256, 128), (1, 4, 2, 640, 640, 64)]


@pytest.mark.parametrize("mod", MODS, ids=["plain", "cap5", "bias", "cap30_bias"])
@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("size", BWD_SIZES, ids=["x".join(map(str, s)) for s in BWD_SIZES])
def test_backward(lib, size, kind, mod):
    B, H, Hkv, Nq, Nkv, d = size
    q, k, v = rand(1, B, H, Nq, d, by=2.0), rand(2, B, Hkv, Nkv, d), rand(3, B, Hkv, Nkv, d)
    dout = rand(4, B, H, Nq, d)
    cap, bias = mod
    m = masks(kind, B, Nq, Nkv)
    sl = slopes_of(H) if bias else None
    if m["kv_lens"] is not None:
        for b in range(B):
            n = int(m["kv_lens"][b])
            k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")
    scale = d ** -0.5
    kw = dict(softcap=cap, alibi_slopes=cuda(sl), key_begin=cuda(m["key_begin"]), key_end=cuda(m["key_end"]),
              kv_lens=cuda(m["kv_lens"]))
    qc, kc, vc = q.cuda(), k.cuda(), v.cuda()
    o, lse = lib.attn_fwd_scoremod(qc, kc, vc, m["causal"], scale, **kw)
    outs = [torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for x in (q, k, v)]
    lib.attn_bwd_scoremod(qc, kc, vc, o, lse, dout.cuda(), m["causal"], scale, dq=outs[0], dk=outs[1], dv=outs[2], **kw)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    ref = (m["causal"], scale, cap, sl, m["key_begin"], m["key_end"], m["kv_lens"])
    want = backward(q, k, v, dout, *ref)
    o64, _, w, t = forward(q, k, v, *ref)
    for name, got, x, tol in zip(("dq", "dk", "dv"), outs, want, grad_bounds(q, k, v, dout, o64, w, t, scale, want)):
        err = (got.cpu().double() - x).abs()
        assert torch.isfinite(got).all(), name
        assert (err <= tol).all(), (name, float(err.max()), float((err / tol).max()))


SHARED_SIZES = [  # key tiles whose steps are shared out: 16 CTAs, several, and more CTAs in all than the GPU holds at once
    (1, 8, 1, 700, 300, 32), (1, 8, 2, 300, 900, 80), (5, 16, 4, 700, 700, 32),
]


@pytest.mark.parametrize("mod", [(0.0, True), (30.0, True)], ids=["bias", "cap30_bias"])
@pytest.mark.parametrize("kind", ["causal", "docs", "window", "empty_rows"])
@pytest.mark.parametrize("size", SHARED_SIZES, ids=["x".join(map(str, s)) for s in SHARED_SIZES])
def test_backward_of_shared_out_key_tiles(lib, size, kind, mod):
    test_backward(lib, size, kind, mod)


def test_backward_of_a_plain_call_equals_the_plain_backward(lib):
    # 192 key tiles fill the GPU: no split of the queries, and the sums run in the plain kernels' order
    q, k, v, g = (rand(20 + i, 4, h, 650, 128).cuda() for i, h in enumerate((16, 8, 8, 16)))
    for causal in (False, True):
        o, lse = lib.attn_fwd_gqa(q, k, v, causal)
        a = lib.attn_bwd(q, k, v, o, lse, g, causal)
        b = lib.attn_bwd_scoremod(q, k, v, o, lse, g, causal)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradients_match_differences():
    """The formula of the backward (and its 64-bit restatement) against central differences of the forward."""
    torch.manual_seed(0)
    B, H, Hkv, Nq, Nkv, d = 1, 2, 1, 5, 7, 32
    q, k, v = (torch.randn(B, h, n, d, dtype=torch.float64) for h, n in ((H, Nq), (Hkv, Nkv), (Hkv, Nkv)))
    g = torch.randn(B, H, Nq, d, dtype=torch.float64)
    kb, ke = documents(B, Nq, Nkv, [3, 4])
    args = (False, 0.3, 2.0, slopes_of(H), kb, ke, torch.tensor([6]))
    got = backward(q, k, v, g, *args)
    loss = lambda: float((forward(q, k, v, *args)[0] * g).sum())  # noqa: E731
    for x, dx in zip((q, k, v), got):
        flat, dflat = x.view(-1), dx.reshape(-1)
        for i in range(0, flat.numel(), 13):
            old, h = float(flat[i]), 1e-5
            flat[i] = old + h
            up = loss()
            flat[i] = old - h
            down = loss()
            flat[i] = old
            assert abs((up - down) / (2 * h) - float(dflat[i])) <= 1e-7


def test_backward_on_another_stream_captured_and_repeated(lib):
    q, k, v, g = (rand(30 + i, 1, h, 400, 64).cuda() for i, h in enumerate((4, 2, 2, 4)))
    kb, ke = (t.cuda() for t in documents(1, 400, 400, [77, 130]))
    kw = dict(softcap=20.0, key_begin=kb, key_end=ke)
    o, lse = lib.attn_fwd_scoremod(q, k, v, True, **kw)
    want = lib.attn_bwd_scoremod(q, k, v, o, lse, g, True, **kw)
    again = lib.attn_bwd_scoremod(q, k, v, o, lse, g, True, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = lib.attn_bwd_scoremod(q, k, v, o, lse, g, True, stream=side, **kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, l2 = lib.attn_fwd_scoremod(q, k, v, True, **kw)
        cap = lib.attn_bwd_scoremod(q, k, v, o2, l2, g, True, **kw)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c, e in zip(want, again, other, cap):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, e)
