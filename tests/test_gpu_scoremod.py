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
        kw["key_begin"][:, ::7] = 2**31 - 1
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
