"""Decode over the 4-bit cache with tensor scales at the ends of their range and a large sum of weights: the output is O / L
times the values' scale, and no step of that leaves fp32's normal numbers before the result does.

One query sees keys of two scores: the first pages that each warp takes score 0, all others 2^a more, under the 2^8 at which
the reference of the weights moves, so that the sum L is as large as it gets.  The sum and a are chosen so that a quotient
scale / L in fp32's subnormal numbers would be 2.4 % off at least (with the largest weight at 1 it lies half way between two)."""
import math

import pytest
import torch

import fp4_ref as F
import paged_ref as R

pytestmark = pytest.mark.gpu
D = 32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def pools():
    """Page 0: keys of zeros; pages 1 .. 63: keys whose dim 0 is 1.  Values positive."""
    k, v = torch.zeros(64, 1, 9 * D, dtype=torch.uint8), torch.zeros(64, 1, 9 * D, dtype=torch.uint8)
    g = torch.Generator().manual_seed(1)
    one = torch.zeros(1, D, dtype=torch.uint8)
    one[0, 0] = 2
    s = torch.full((1, D // 16), 0x38, dtype=torch.uint8)  # 1.0
    for page in range(64):
        for t in range(16):
            if page:
                F.write(k, page, t, one, s, False)
            F.write(v, page, t, torch.randint(1, 8, (1, D), generator=g).to(torch.uint8), s, True)
    return k, v


def two_levels(n, run):
    """A table row of n pages whose first two of each `run` pages are page 0."""
    row = 1 + torch.arange(n, dtype=torch.int32) % 63
    row[torch.arange(n) % run < 2] = 0
    return row


def decode(lib, k, v, table, tokens, scale, ks, vs):
    B = table.shape[0]
    q = torch.zeros(B, 1, D, dtype=torch.bfloat16)
    q[..., 0] = 1
    ctx = torch.full((B,), tokens, dtype=torch.int32)
    out = lib.paged_attn_decode_fp4(q.cuda(), k.cuda(), v.cuda(), ks, vs, table.cuda(), ctx.cuda(), scale=scale)
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    return out


# a: of the sums 14336 2^a + 2048 and 16256 2^a + 128, 20.5 times (scale / 2^-149)^-1 each
@pytest.mark.parametrize("rows, run, a", [(1, 16, 7.923), (1824, 256, 7.742)], ids=["cluster", "whole_rows"])
@pytest.mark.parametrize("vs", [1e-37, 3e34, 1e-3])
@pytest.mark.parametrize("ks", [1e-37, 1e37])
def test_rows_of_one_cta_or_cluster(lib, rows, run, a, vs, ks):
    k, v = pools()
    row = two_levels(1024, run)
    scale = a * math.log(2.0) / ks
    out = decode(lib, k, v, row.repeat(rows, 1), 16384, scale, ks, vs)
    want = R.decode(torch.eye(D)[:1][None].to(torch.bfloat16), F.read(k, False), F.read(v, True), row[None], [16384], scale * ks)
    R.check((out[0].cpu().double() / vs).float(), out[1].cpu(), *(t.expand(rows, *t.shape[1:]) for t in want))


@pytest.mark.parametrize("vs", [1e-37, 3e34])
def test_rows_of_many_ctas(lib, vs):
    # 8394752 tokens of one score: scale / L would be 8.5 times 2^-149
    k, v = pools()
    row = 1 + torch.arange(64 * 8198, dtype=torch.int32) % 63
    n = 63 * 8328  # whole turns of the 63 pages
    out = decode(lib, k, v, row[None], 16 * n, 1e-3, 1.0, vs)
    want = R.decode(torch.eye(D)[:1][None].to(torch.bfloat16), F.read(k, False), F.read(v, True), row[None, :63], [16 * 63], 1e-3)
    # (LSE: ln 8328 more, its sum a chain of roundings as in the test of 2^24 tokens: 3e-4)
    assert (out[1].cpu().double() - want[1] - math.log(8328)).abs().max() <= 3e-4
    R.check((out[0].cpu().double() / vs).float(), want[1].float(), *want)
