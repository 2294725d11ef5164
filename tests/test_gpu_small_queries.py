"""Decode with modified scores and over shared prefixes, e4m3 cache, with queries far below 1: each head is rounded to f16
after a power of two of its own, up as well as down (bounds in paged_ref.check: what the rounding leaves out is at most 2^-18
of a head's largest value)."""
import pytest
import torch

import paged_ref as R
from test_gpu_decode_scoremod import FORMS, make, run, slopes_of
from test_gpu_decode_shared import make as make_shared
from test_gpu_small_queries_fp4 import IDS, SHAPES, less

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


@pytest.mark.parametrize("mod", [(0.0, False), (5.0, False), (0.0, True)], ids=["plain", "cap", "bias"])
@pytest.mark.parametrize("by", [2.0 ** -20, 2.0 ** -100], ids=["2^-20", "2^-100"])
@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_modified_scores(lib, shape, spare, by, mod):
    H, Hkv, d, ctx = shape
    cap, bias = mod
    x = less(make(len(ctx), H, Hkv, d, ctx, True, 3, None, spare), by)
    sl, scale = slopes_of(H) if bias else None, d ** -0.5 / by
    out = run(lib, x, True, scale=scale, softcap=cap, alibi_slopes=sl)
    R.check(out[0].cpu(), out[1].cpu(), *R.decode(x[0], x[1], x[2], x[3], ctx, scale, True, cap, sl))


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_scores_that_vanish(lib, shape):
    H, Hkv, d, ctx = shape
    x = less(make(len(ctx), H, Hkv, d, ctx, True, 4), 2.0 ** -125)
    for scale in (d ** -0.5, 1e-30):
        out = run(lib, x, True, scale=scale)
        R.check(out[0].cpu(), out[1].cpu(), *R.decode(x[0], x[1], x[2], x[3], ctx, scale, True))


def test_shared_prefixes(lib):
    by, scale = 2.0 ** -25, 64 ** -0.5 * 2.0 ** 25
    x = make_shared(8, 2, 64, 2, [10, 3], [200, 190, 60, 77], True, 4, spare=1)
    x["q"] = (x["q"].float() * by).to(torch.bfloat16)
    got = lib.paged_attn_decode_shared_fp8(*(x[n].cuda() for n in ("q", "k", "v")), 0.02, 0.02,
                                           *(x[n].cuda() for n in ("table", "ctx", "shared")), 2, scale=scale)
    R.check(got[0].cpu(), got[1].cpu(), *R.decode(x["q"], x["k"], x["v"], x["full"], x["ctx"].tolist(), scale, True))
