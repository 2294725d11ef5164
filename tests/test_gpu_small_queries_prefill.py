"""Chunked prefill over an e4m3 cache, and shared pages read once per group, with queries far below 1: each row is rounded to
f16 after a power of two of its own, up as well as down (bounds in paged_ref.check: what the rounding leaves out is at most
2^-18 of a row's largest value)."""
import pytest
import torch

import paged_ref as R
from test_gpu_decode_scoremod import make
from test_gpu_decode_shared import make as make_shared, wide
from test_gpu_small_queries_fp4 import less

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def finite(x):
    x = list(x)
    for t in x[1:3]:
        t[t == 0x7F] = 0
    return x


@pytest.mark.parametrize("by", [2.0 ** -8, 2.0 ** -20, 2.0 ** -60], ids=["2^-8", "2^-20", "2^-60"])
@pytest.mark.parametrize("shape", [(4, 4, 64, 33, [300, 17]), (8, 2, 128, 140, [90, 700]), (6, 1, 32, 1, [1, 200]), (2, 2, 80, 70, [130])],
                         ids=lambda s: f"H{s[0]}kv{s[1]}d{s[2]}N{s[3]}")
def test_prefill(lib, shape, by):
    H, Hkv, d, N, ctx = shape
    x = less(finite(make(len(ctx), H * N, Hkv, d, ctx, True, 3)), by)  # (the rows of a head as heads of its group: no causal mask)
    q, k, v, table, lens = (t.cuda() for t in x)
    for scale in (d ** -0.5 / by, d ** -0.5):  # (with the second the scores vanish)
        o, lse = lib.paged_attn_prefill_fp8(q.view(len(ctx), H, N, d), k, v, 0.02, 0.02, table, lens, False, scale=scale)
        R.check(o.cpu().view(x[0].shape), lse.cpu().view(len(ctx), H * N), *R.decode(x[0], x[1], x[2], x[3], ctx, scale, True))


def test_prefill_rows_of_several_magnitudes(lib):
    H, d, N, ctx = 2, 64, 50, [400]
    x = finite(make(1, H * N, 2, d, ctx, True, 5))
    x[0] = (x[0].float() * torch.tensor([2.0 ** -(10 + i % 4) for i in range(H * N)])[:, None]).to(torch.bfloat16)
    q, k, v, table, lens = (t.cuda() for t in x)
    scale = d ** -0.5 * 2.0 ** 11
    o, lse = lib.paged_attn_prefill_fp8(q.view(1, H, N, d), k, v, 0.02, 0.02, table, lens, False, scale=scale)
    R.check(o.cpu().view(x[0].shape), lse.cpu().view(1, H * N), *R.decode(x[0], x[1], x[2], x[3], ctx, scale, True))


@pytest.mark.parametrize("by", [2.0 ** -20, 2.0 ** -60], ids=["2^-20", "2^-60"])
def test_shared_pages_read_once(lib, by):
    c = (8, 2, 64, 2, [10, 3], [200, 190, 60, 77])
    x = make_shared(*c, True, 4, spare=2 * wide(*c))
    x["q"] = (x["q"].float() * by).to(torch.bfloat16)
    scale = 64 ** -0.5 / by
    got = lib.paged_attn_decode_shared_fp8(*(x[n].cuda() for n in ("q", "k", "v")), 0.02, 0.02,
                                           *(x[n].cuda() for n in ("table", "ctx", "shared")), 2, scale=scale)
    R.check(got[0].cpu(), got[1].cpu(), *R.decode(x["q"], x["k"], x["v"], x["full"], x["ctx"].tolist(), scale, True))
