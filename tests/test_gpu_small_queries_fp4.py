"""Decode over the 4-bit cache with queries far below 1: each head is rounded to f16 after a power of two of its own, up as
well as down (bounds in paged_ref.check: what the rounding leaves out is at most 2^-18 of a head's largest value)."""
import pytest
import torch

import paged_ref as R
from test_gpu_decode_fp4 import make, run, want
from test_gpu_decode_scoremod import FORMS, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


SHAPES = [(12, 2, 80, [300, 17, 1025]), (16, 1, 128, [90, 700]), (4, 4, 32, [1, 33]), (40, 2, 64, [130, 0])]
IDS = [f"H{s[0]}kv{s[1]}d{s[2]}" for s in SHAPES]


def less(x, by):
    """The queries times `by` (a power of two), one of them all zeros."""
    x = list(x)
    q = x[0].clone()
    q[0, 1] = 0
    x[0] = (q.float() * by).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("mod", [(0.0, False), (5.0, False), (0.0, True), (30.0, True)], ids=["plain", "cap", "bias", "cap_bias"])
@pytest.mark.parametrize("by", [2.0 ** -8, 2.0 ** -20, 2.0 ** -30, 2.0 ** -100], ids=["2^-8", "2^-20", "2^-30", "2^-100"])
@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_small_queries_and_a_large_scale(lib, shape, spare, by, mod):
    H, Hkv, d, ctx = shape
    cap, bias = mod
    x = less(make(len(ctx), H, Hkv, d, ctx, 3, None, spare), by)
    sl, scale = slopes_of(H) if bias else None, d ** -0.5 / by
    out = run(lib, x, scale=scale, softcap=cap, alibi_slopes=sl)
    R.check(out[0].cpu(), out[1].cpu(), *want(x, scale, cap, sl))


@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_queries_at_the_end_of_bf16(lib, shape, spare):
    H, Hkv, d, ctx = shape
    x = less(make(len(ctx), H, Hkv, d, ctx, 4, None, spare), 2.0 ** -125)  # many of them subnormal
    for scale in (d ** -0.5 * 2.0 ** 125, d ** -0.5, 1e-30):  # (the last two: all scores are 0 to fp32)
        out = run(lib, x, scale=scale)
        R.check(out[0].cpu(), out[1].cpu(), *want(x, scale))
    out = run(lib, x, scale=d ** -0.5, softcap=20.0, alibi_slopes=slopes_of(H))
    R.check(out[0].cpu(), out[1].cpu(), *want(x, d ** -0.5, 20.0, slopes_of(H)))


def test_heads_of_several_magnitudes(lib):
    # each head by a factor of its own; the common scale keeps the scores of most of them in the range that weights show
    x = list(make(3, 16, 2, 64, [200, 77, 900], 5))
    by = torch.tensor([2.0 ** -(10 + h % 4) for h in range(16)])
    x[0] = (x[0].float() * by[:, None]).to(torch.bfloat16)
    scale = 64 ** -0.5 * 2.0 ** 11
    out = run(lib, x, scale=scale)
    R.check(out[0].cpu(), out[1].cpu(), *want(x, scale))
