"""A paged cache with everything unused set to NaN, and decode over it in 64 bits (CPU), for the tests."""
import torch

PS = 16


def cache(tables_pages, Hkv, d, seed, fp8=False):
    """Pools of `n` pages of random values (e4m3 codes when fp8) plus one page of NaN; returns k, v, nan page id."""
    g = torch.Generator().manual_seed(seed)
    n = tables_pages + 1
    k, v = (torch.randn(n, Hkv, PS, d, generator=g).to(torch.bfloat16) for _ in range(2))
    if fp8:
        k, v = ((t.float() / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for t in (k, v))
        k[-1], v[-1] = 0x7F, 0x7F
    else:
        k[-1], v[-1] = float("nan"), float("nan")
    return k, v, n - 1


def poison(k, v, page, first, last, fp8):
    """Slots first <= i < last of a page become NaN."""
    for t in (k, v):
        t[page, :, first:last] = 0x7F if fp8 else float("nan")


def values(t, fp8):
    return t.view(torch.float8_e4m3fn).double() * 0.02 if fp8 else t.double()


def tokens(k, v, row, lo, hi, fp8):
    """Keys and values [n, Hkv, d] of the mapped tokens lo <= j < hi of a table row, and their positions."""
    j = torch.arange(max(lo, 0), max(hi, lo, 0))
    page = row.long()[j // PS]
    ok = (page >= 0) & (page < k.shape[0])
    j, page = j[ok], page[ok]
    return values(k[page, :, j % PS], fp8), values(v[page, :, j % PS], fp8), j


def decode(q, k, v, table, ctx, scale, fp8=False, softcap=0.0, slopes=None, begin=None):
    """o [B,H,d], lse [B,H] and W|v| [B,H,d] in float64."""
    B, H, d = q.shape
    Hkv = k.shape[1]
    o, wv = torch.zeros(B, H, d, dtype=torch.float64), torch.zeros(B, H, d, dtype=torch.float64)
    lse = torch.full((B, H), float("-inf"), dtype=torch.float64)
    for b in range(B):
        hi = min(max(int(ctx[b]), 0), table.shape[1] * PS)
        lo = 0 if begin is None else int(begin[b])
        kk, vv, j = tokens(k, v, table[b], lo, hi, fp8)
        if len(j) == 0:
            continue
        kk, vv = (t.permute(1, 0, 2).repeat_interleave(H // Hkv, 0) for t in (kk, vv))
        x = torch.einsum("hd,hnd->hn", q[b].double(), kk) * scale
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        if slopes is not None:
            x = x - slopes.double()[:, None] * (hi - 1 - j).double()
        lse[b] = torch.logsumexp(x, -1)
        w = torch.softmax(x, -1)
        o[b], wv[b] = torch.einsum("hn,hnd->hd", w, vv), torch.einsum("hn,hnd->hd", w, vv.abs())
    return o, lse, wv


def check(o, lse, want, wl, wv):
    """The bounds: weights rounded once to bf16 or f16 (2^-8 at most), O once (2^-8); a score is d <= 128 exact
    products summed in fp32, off by at most 128 * 2^-23 scale sum |q k| (about 14 here: 2e-4), which moves
    weights and their sum by that; 1 % for the cross terms.  LSE: the scores' error averages over random
    signs: 1e-4."""
    err = (o.double() - want).abs()
    tol = 1.01 * ((2.0 ** -8 + 4e-4) * wv + 2.0 ** -8 * want.abs()) + 1e-30
    assert torch.isfinite(o).all()
    assert (err <= tol).all(), float((err / tol).max())
    assert torch.equal(torch.isneginf(lse.double()), torch.isneginf(wl))
    assert (lse.double() - wl).nan_to_num(0.0).abs().max() <= 1e-4
    assert (o[torch.isneginf(wl)] == 0).all()
