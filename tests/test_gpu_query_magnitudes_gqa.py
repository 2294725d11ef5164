"""paged_attn_decode_fp8 with query heads of very different magnitudes in one group: each query is rounded to f16
after a power of two of its own (bounds in paged_ref.check)."""
import pytest
import torch

import paged_ref as R
from test_gpu_decode_scoremod import make
from test_gpu_query_magnitudes import enlarge, ordinary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


SHAPES = [(4, 1, 64, [300, 17], [2]), (8, 1, 128, [90, 700], [0, 7]), (16, 1, 32, [1, 200], [3, 12]), (40, 2, 80, [130], [5, 39]),
          (12, 2, 96, [1500, 48, 33], [11])]


@pytest.mark.parametrize("by", [2.0 ** 16, 2.0 ** 40, 2.0 ** 110], ids=["2^16", "2^40", "2^110"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"H{s[0]}kv{s[1]}d{s[2]}" for s in SHAPES])
def test_grouped_decode(lib, shape, by):
    H, Hkv, d, ctx, huge = shape
    x = list(make(len(ctx), H, Hkv, d, ctx, True, 3))
    x[0] = enlarge(x[0], huge, by)
    q, k, v, table, lens = (t.cuda() for t in x)
    got = lib.paged_attn_decode_fp8(q, k, v, 0.02, 0.02, table, lens)
    ordinary(got, R.decode(x[0], x[1], x[2], x[3], ctx, d ** -0.5, True), huge)
