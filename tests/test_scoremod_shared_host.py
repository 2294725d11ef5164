"""Host-side refusals and workspace sizes of attention with modified scores and of the shared-pages decode:
bad arguments come back as a status before any device work."""
import pytest

A = 1 << 20  # fake, 16-byte aligned addresses: the checks fail before any use
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from attn_fwd_02_gb300 import binding
    from attn_fwd_02_gb300 import build as buildmod
    buildmod.build()
    return binding.load_library()


def fwd(lib, q=A, k=A, v=A, o=A, lse=None, B=1, Hq=4, Hkv=2, Nq=10, Nkv=20, d=64, causal=0, scale=0.1, cap=0.0,
        slopes=None, begin=None, end=None, lens=None):
    return lib.attn_fwd_scoremod(q, k, v, o, lse, B, Hq, Hkv, Nq, Nkv, d, causal, scale, cap, slopes, begin, end, lens, None)


def bwd(lib, q=A, k=A, v=A, o=A, lse=A, g=A, dq=A, dk=A, dv=A, B=1, Hq=4, Hkv=2, Nq=10, Nkv=20, d=64, causal=0, scale=0.1,
        cap=0.0, slopes=None, begin=None, end=None, lens=None, ws=A, n=1 << 20):
    return lib.attn_bwd_scoremod(q, k, v, o, lse, g, dq, dk, dv, B, Hq, Hkv, Nq, Nkv, d, causal, scale, cap, slopes, begin,
                                 end, lens, ws, n, None)


COMMON = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(B=0), 1), (dict(Hkv=3), 1),
    (dict(Nq=0), 1), (dict(Nkv=-1), 1), (dict(causal=2), 1), (dict(scale=0.0), 1), (dict(scale=INF), 1),
    (dict(cap=-1.0), 1), (dict(cap=NAN), 1), (dict(cap=INF), 1), (dict(cap=1e31), 1), (dict(cap=1e-32, scale=1.0), 1),
    (dict(d=48), 2), (dict(d=256), 2), (dict(q=A + 8), 3), (dict(slopes=A + 2), 3), (dict(begin=A + 1), 3),
    (dict(end=A + 2), 3), (dict(lens=A + 3), 3),
]


@pytest.mark.parametrize("bad, status", COMMON + [(dict(lse=A + 2), 3)])
def test_forward_refusals(lib, bad, status):
    assert fwd(lib, **bad) == status


@pytest.mark.parametrize("bad, status", COMMON + [
    (dict(lse=None), 1), (dict(g=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1), (dict(g=A + 8), 3),
    (dict(dk=A + 4), 3), (dict(ws=None), 4), (dict(ws=A + 8), 4), (dict(n=64), 4)])
def test_backward_refusals(lib, bad, status):
    assert bwd(lib, **bad) == status


def decode(lib, q=A, k=A, v=A, table=A, ctx=A, ps=16, o=A, lse=None, B=2, H=4, Hkv=2, d=64, pages=8, pool=9, scale=0.1,
           cap=0.0, slopes=None, begin=None, ws=A, n=1 << 30, scales=None):
    if scales is None:
        return lib.paged_attn_decode_scoremod(q, k, v, table, ctx, ps, o, lse, B, H, Hkv, d, pages, pool, scale, cap, slopes,
                                              begin, ws, n, None)
    return lib.paged_attn_decode_scoremod_fp8(q, k, v, *scales, table, ctx, ps, o, lse, B, H, Hkv, d, pages, pool, scale, cap,
                                              slopes, begin, ws, n, None)


def shared(lib, q=A, k=A, v=A, table=A, ctx=A, sp=A, S=2, ps=16, o=A, lse=None, B=4, H=4, Hkv=2, d=64, pages=8, pool=9,
           scale=0.1, ws=A, n=1 << 30, scales=None):
    if scales is None:
        return lib.paged_attn_decode_shared(q, k, v, table, ctx, sp, S, ps, o, lse, B, H, Hkv, d, pages, pool, scale, ws, n, None)
    return lib.paged_attn_decode_shared_fp8(q, k, v, *scales, table, ctx, sp, S, ps, o, lse, B, H, Hkv, d, pages, pool, scale,
                                            ws, n, None)


PAGED = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(table=None), 1), (dict(ctx=None), 1), (dict(o=None), 1), (dict(B=0), 1),
    (dict(H=5), 1), (dict(Hkv=0), 1), (dict(pages=0), 1), (dict(pool=0), 1), (dict(scale=-1.0), 1), (dict(scale=NAN), 1),
    (dict(pages=1 << 28), 1), (dict(pool=1 << 30, Hkv=4), 1), (dict(d=72), 2), (dict(ps=32), 2), (dict(q=A + 2), 3),
    (dict(table=A + 1), 3), (dict(lse=A + 2), 3), (dict(ws=None), 4), (dict(ws=A + 4), 4), (dict(n=100), 4),
    (dict(scales=(0.0, 1.0)), 1), (dict(scales=(1.0, INF)), 1), (dict(scales=(1e38, 1.0), scale=100.0), 1),
]


@pytest.mark.parametrize("bad, status", PAGED + [
    (dict(cap=-2.0), 1), (dict(cap=NAN), 1), (dict(cap=2e30), 1), (dict(slopes=A + 1), 3), (dict(begin=A + 2), 3),
    (dict(B=1 << 16), 1), (dict(B=65535, H=65535, Hkv=1), 1)])
def test_decode_refusals(lib, bad, status):
    assert decode(lib, **bad) == status


@pytest.mark.parametrize("bad, status", PAGED + [
    (dict(sp=None), 1), (dict(S=0), 1), (dict(S=3), 1), (dict(S=-2), 1), (dict(sp=A + 2), 3),
    (dict(B=65534, H=65535, Hkv=1), 1)])
def test_shared_refusals(lib, bad, status):
    assert shared(lib, **bad) == status


def test_workspace_sizes(lib):
    ws = lib.paged_attn_decode_scoremod_workspace_size
    assert ws(32, 32, 8, 128, 512, 16) == 32 * 32 * 8 * (128 + 4) * 4      # a full batch: splits of 64 pages
    assert ws(1, 8, 8, 64, 512, 16) == 8 * 64 * (64 + 4) * 4               # a small one: of 8
    assert ws(1, 8, 8, 64, 1, 16) == 8 * (64 + 4) * 4
    assert ws(1, 8, 3, 64, 1, 16) == 0 and ws(1, 8, 8, 48, 1, 16) == 0 and ws(1, 8, 8, 64, 1, 32) == 0
    sh = lib.paged_attn_decode_shared_workspace_size
    for args in ((4, 12, 12, 64, 36, 4, 16), (32, 32, 8, 128, 544, 32, 16), (128, 32, 8, 128, 1087, 64, 16),
                 (2, 130, 1, 32, 8, 2, 16), (3, 8, 2, 80, 5, 1, 16), (4096, 64, 8, 128, 100, 2, 16)):
        n = sh(*args)
        assert n > 0 and n % (args[0] * args[1] * (args[3] + 4) * 4) == 0, args
    assert sh(4, 8, 2, 64, 8, 3, 16) == 0 and sh(4, 8, 2, 64, 8, 0, 16) == 0 and sh(4, 8, 2, 40, 8, 2, 16) == 0
    bw = lib.attn_bwd_scoremod_workspace_size
    assert bw(2, 16, 16, 8192, 8192, 128) == 2 * 16 * 8192 * 4 + 2 * 64 * 8        # no split: row term and intervals
    assert bw(2, 16, 4, 1000, 1000, 64) > 2 * 16 * 1000 * 4 + 2 * 8 * 8 + 2 * 2 * 2 * 4 * 1000 * 64 * 4
    assert bw(0, 1, 1, 1, 1, 32) == 0 and bw(1, 4, 3, 1, 1, 32) == 0
