"""Chunked prefill over pages whose slots past the sequence's last token were never written: they may hold anything (NaN, inf),
as in the decodes.  A cache of bf16, of e4m3, and 4-bit pages brought back as bf16 (bounds in paged_ref.check)."""
import pytest
import torch

import fp4_ref as F
import paged_ref as R
from test_gpu_decode_fp4 import KS, VS, make as make4
from test_gpu_decode_scoremod import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def want(q, k, v, table, ctx, scale, causal, fp8):
    """q [B, H, N, d]; row i of a sequence as a sequence of its own, of the tokens that it sees."""
    B, H, N, d = q.shape
    rows = q.permute(0, 2, 1, 3).reshape(B * N, H, d)
    seen = [max(0, c - N + i + 1) if causal else c for c in ctx for i in range(N)]
    out = R.decode(rows, k, v, table.repeat_interleave(N, 0), seen, scale, fp8)
    return [t.view(B, N, H, *t.shape[2:]).transpose(1, 2) for t in out]


SHAPES = [(4, 4, 64, 33, [300, 17, 64]), (8, 2, 128, 140, [290, 701]), (6, 1, 32, 1, [1, 200, 0]), (2, 2, 80, 70, [130, 129, 15]), (4, 1, 96, 270, [271])]
IDS = [f"H{s[0]}kv{s[1]}d{s[2]}N{s[3]}" for s in SHAPES]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("cache", ["bf16", "inf", "e4m3", "fp4"])
def test_last_pages_never_written(lib, shape, causal, cache):
    H, Hkv, d, N, ctx = shape
    B, scale = len(ctx), d ** -0.5
    if cache == "fp4":
        _, k4, v4, table, lens = make4(B, 2 * Hkv, Hkv, d, ctx, 3)
        k, v = (F.read(t, s).float() * x for t, s, x in ((k4, False, KS), (v4, True, VS)))
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        ids = torch.arange(k4.shape[0], dtype=torch.int32).cuda()
        kd, vd = lib.paged_kv_unpack_fp4(k4.cuda(), v4.cuda(), KS, VS, ids)
        assert kd.isnan().any() and vd.isnan().any()
    else:
        _, k, v, table, lens = make(B, 2 * Hkv, Hkv, d, ctx, cache == "e4m3", 3)
        if cache == "inf":
            k, v = (torch.where(t.isnan(), float("inf"), t) for t in (k, v))
        kd, vd = k.cuda(), v.cuda()
    q = (torch.randn(B, H, N, d, generator=torch.Generator().manual_seed(2)) * 2).to(torch.bfloat16)
    f, scales = (lib.paged_attn_prefill_fp8, (0.02, 0.02)) if cache == "e4m3" else (lib.paged_attn_prefill, ())
    o, lse = f(q.cuda(), kd, vd, *scales, table.cuda(), lens.cuda(), causal, scale=scale)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    R.check(o.cpu(), lse.cpu(), *want(q, k, v, table, ctx, scale, causal, cache == "e4m3"))
