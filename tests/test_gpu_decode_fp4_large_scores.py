"""Decode over the 4-bit cache with scores far past those whose differences matter: the tokens of the largest score share the
weight evenly, the others have none, and nothing overflows on the way (bounds in paged_ref.check; LSE to fp32's rounding of it)."""
import pytest
import torch

import fp4_ref as F
import paged_ref as R
from test_gpu_decode_scoremod import FORMS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


@pytest.mark.parametrize("bias", [False, True], ids=["plain", "modified"])
@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("d, group, n", [(32, 1, 9), (64, 3, 300), (128, 8, 700), (80, 16, 130)])
@pytest.mark.parametrize("size", [1e3, 3e6, 7e7, 1.1e9, 1e13, 1e20, 1e30])
def test_the_largest_share_the_weight(lib, d, group, n, spare, bias, size):
    g = torch.Generator().manual_seed(n)
    pages = (n + 15) // 16
    k, v = (torch.zeros(pages, 1, 9 * d, dtype=torch.uint8) for _ in range(2))
    s = torch.full((1, d // 16), 0x38, dtype=torch.uint8)  # 1.0
    for t in range(n):
        codes = torch.zeros(1, d, dtype=torch.uint8)
        codes[0, 0] = torch.randint(0, 8, (1,), generator=g)  # ascending and descending, with ties
        if t % 50 == 0:
            codes[0, 0] = 7
        F.write(k, t // 16, t % 16, codes, s, False)
        F.write(v, t // 16, t % 16, torch.randint(0, 16, (1, d), generator=g).to(torch.uint8), s, True)
    q = torch.zeros(1, group, d, dtype=torch.bfloat16)
    q[:, :, 0] = 1.5
    scale = size / 9  # the largest score: 1.5 * 6 * scale
    table = torch.full((1, pages + spare), -1, dtype=torch.int32)
    table[0, :pages] = torch.arange(pages)
    out = lib.paged_attn_decode_fp4(q.cuda(), k.cuda(), v.cuda(), 1.0, 1.0, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                    scale=scale, alibi_slopes=torch.zeros(group).cuda() if bias else None)
    o, lse, wv = R.decode(q, F.read(k, False), F.read(v, True), table, [n], scale)
    err = (out[0].cpu().double() - o).abs()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1]).all()
    assert (err <= 1.01 * ((2.0 ** -8 + 4e-4) * wv + 2.0 ** -8 * o.abs()) + 1e-30).all()
    # (the score, its product with the scale and log2 e, the reference, the sum and ln 2: a few roundings of 2^-24)
    assert ((out[1].cpu().double() - lse).abs() <= 1e-4 + 8 * 2.0 ** -24 * lse.abs()).all()
