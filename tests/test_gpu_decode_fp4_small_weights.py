"""Decode over the 4-bit cache where what counts is the small weights: the tokens of large weight have values of exactly 0, which 4
bits often have.  A weight from 2^-21 of the largest on is rounded to f16's 11 bits, smaller ones are off by 2^-32 of the largest at
most; the rest of the bound is paged_ref.check's."""
import math

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


@pytest.mark.parametrize("cap", [0.0, 40.0])
@pytest.mark.parametrize("spare", **FORMS)
@pytest.mark.parametrize("d, n", [(32, 9), (64, 300), (128, 40), (80, 16)])
@pytest.mark.parametrize("bits", [10, 14, 17, 20, 24])
def test_values_of_zero_under_the_large_weights(lib, d, n, spare, cap, bits):
    g = torch.Generator().manual_seed(bits)
    pages = (n + 15) // 16
    k, v = (torch.zeros(pages, 1, 9 * d, dtype=torch.uint8) for _ in range(2))
    s = torch.full((1, d // 16), 0x38, dtype=torch.uint8)  # 1.0
    for t in range(n):
        large = t % 7 == 3
        codes = torch.zeros(1, d, dtype=torch.uint8)
        codes[0, 0] = 6 if large else 2          # a score of 4 or of 1
        codes[0, 1] = 0 if large else t % 2 + 1  # .. and up to 1/8 more
        F.write(k, t // 16, t % 16, codes, s, False)
        F.write(v, t // 16, t % 16, torch.zeros(1, d, dtype=torch.uint8) if large else torch.randint(1, 8, (1, d), generator=g).to(torch.uint8), s, True)
    q = torch.zeros(1, 2, d, dtype=torch.bfloat16)
    q[:, :, 0], q[:, :, 1] = 1.0, 0.125
    scale = bits * math.log(2.0) / 3  # the small weights: 2^-bits of the large ones, and a little more
    table = torch.full((1, pages + spare), -1, dtype=torch.int32)
    table[0, :pages] = torch.randperm(pages, generator=g).int()
    order = table[0, :pages].long()
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    kk[order], vv[order] = k, v
    out = lib.paged_attn_decode_fp4(q.cuda(), kk.cuda(), vv.cuda(), 1.0, 1.0, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                    scale=scale, softcap=cap)
    o, lse, wv = R.decode(q, F.read(kk, False), F.read(vv, True), table, [n], scale, False, cap)
    most = 6.0 * n * 2.0 ** -32  # of a weight under 2^-21, times the largest value
    err = (out[0].cpu().double() - o).abs()
    tol = 1.01 * ((2.0 ** -8 + 4e-4) * wv + 2.0 ** -8 * o.abs()) + (most if bits > 18 else 0.0)
    assert (err <= tol).all(), float((err / tol).max())
    assert (out[1].cpu().double() - lse).abs().max() <= 1e-4
