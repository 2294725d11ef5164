"""The rotation on the way into the 4-bit cache rounds as the rotation alone does: fp32 fma(x, c, -(y s)) and fma(y, c, x s), the
second product rounded once, the queries to bf16 once, the keys quantised from fp32."""
import pytest
import torch

import fp4_ref as F
from test_gpu_append_rope import angles

pytestmark = pytest.mark.gpu
KS, VS = 0.0113, 0.37


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def turned(x, pos, pair, cs, inter):
    """x [B, heads, N, d] turned in fp32.  A product of bf16 and fp32 has 32 bits, exact in float64, and so is its sum with the
    rounded one but for exponents 20 apart, where the smaller only breaks ties."""
    r = cs.shape[1]
    i = torch.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    row = pos[torch.tensor(list(pair))].permute(1, 2, 0)
    c, s = cs[row, i][:, None], cs[row, r // 2 + i][:, None]
    f, out = x.float(), x.float()
    xa, xb = f[..., a], f[..., b]
    out[..., a] = (xa.double() * c.double() - (xb * s).double()).float()
    out[..., b] = (xb.double() * c.double() + (xa * s).double()).float()
    return out


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("d, r", [(32, 16), (64, 64), (80, 80), (96, 48), (128, 128)])
def test_queries_and_codes_bit_for_bit(lib, d, r, inter):
    B, H, Hkv, N, A = 2, 5, 3, 37, 3
    g = torch.Generator().manual_seed(11)
    qkv = torch.randn(B, N, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda().transpose(1, 2)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    pos, cs = torch.randint(0, 50, (A, B, N), generator=g), angles(50, r)
    pair = bytes(torch.randint(0, A, (r // 2,), generator=g).tolist())
    start = torch.tensor([0, 5], dtype=torch.int32)
    table = torch.randperm(8, generator=g).view(2, 4).int()
    pools = [torch.zeros(8, Hkv, 9 * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = lib.paged_kv_append_fp4(q, k, v, *pools, KS, VS, table.cuda(), start.cuda(), cos_sin=cs.cuda(),
                                  positions=pos.int().cuda(), pair_axis=pair, interleaved=inter)
    alone = lib.attn_rope_axes(q, None, cs.cuda(), pos.int().cuda(), pair, inter)[0]
    assert torch.equal(out, alone)
    assert torch.equal(out.cpu(), turned(q.cpu(), pos, pair, cs, inter).to(torch.bfloat16))
    codes, scales = F.quantise(turned(k.cpu(), pos, pair, cs, inter), KS)
    want = torch.zeros(8, Hkv, 9 * d, dtype=torch.uint8)
    for b in range(B):
        for t in range(N):
            at = int(start[b]) + t
            F.write(want, int(table[b, at // 16]), at % 16, codes[b, :, t], scales[b, :, t], False)
    assert torch.equal(pools[0].cpu(), want)
