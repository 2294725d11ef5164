"""paged_attn_decode_fp8 with queries far below 1: each head is rounded to f16 after a power of two of its own, up as well as
down (bounds in paged_ref.check: what the rounding leaves out is at most 2^-18 of a head's largest value)."""
import pytest
import torch

import paged_ref as R
from test_gpu_decode_scoremod import make
from test_gpu_small_queries_fp4 import less

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


SHAPES = [(4, 4, 64, [300, 17]), (8, 1, 128, [90, 700]), (16, 1, 32, [1, 200]), (40, 2, 80, [130]), (12, 2, 96, [1500, 48, 33])]


@pytest.mark.parametrize("by", [2.0 ** -20, 2.0 ** -60], ids=["2^-20", "2^-60"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"H{s[0]}kv{s[1]}d{s[2]}" for s in SHAPES])
def test_grouped_decode(lib, shape, by):
    H, Hkv, d, ctx = shape
    x = less(make(len(ctx), H, Hkv, d, ctx, True, 3), by)
    q, k, v, table, lens = (t.cuda() for t in x)
    for scale in (d ** -0.5 / by, d ** -0.5):  # (with the second the scores vanish)
        got = lib.paged_attn_decode_fp8(q, k, v, 0.02, 0.02, table, lens, scale=scale)
        R.check(got[0].cpu(), got[1].cpu(), *R.decode(x[0], x[1], x[2], x[3], ctx, scale, True))
