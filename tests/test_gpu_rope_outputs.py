"""Outputs of the rotation by several axes: every order of the dims and every gap between rows gives what a dense output gets,
and what lies between the rows stays; expanded outputs are refused."""
import itertools

import pytest
import torch

from test_gpu_append_rope import angles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def args(B, H, N, d, g):
    q = torch.randn(B, H, N, d, generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 40, (2, B, N), generator=g).int().cuda()
    return q, angles(40, d).cuda(), pos, bytes([0, 1] * (d // 4))


@pytest.mark.parametrize("sizes", [(2, 3, 5), (1, 4, 7), (3, 1, 2), (2, 2, 1), (1, 1, 1)])
@pytest.mark.parametrize("order", list(itertools.permutations(range(3))), ids=str)
def test_every_order_of_the_dims(lib, sizes, order):
    d, gap = 64, 8
    q, *rest = args(*sizes, d, torch.Generator().manual_seed(3))
    want = lib.attn_rope_axes(q, None, *rest)[0]
    for inner in (d, d + gap):
        base = torch.full((*(sizes[i] for i in order), inner), 3.0, dtype=torch.bfloat16, device="cuda")
        out = base[..., :d].permute(*(order.index(i) for i in range(3)), 3)
        got = lib.attn_rope_axes(q, None, *rest, q_out=out)[0]
        assert got is out and torch.equal(out, want) and (base[..., d:] == 3).all()


def test_expanded_outputs_are_refused(lib):
    q, *rest = args(2, 3, 5, 64, torch.Generator().manual_seed(4))
    for shape in ((1, 3, 5), (2, 1, 5), (2, 3, 1)):
        one = torch.zeros(*shape, 64, dtype=torch.bfloat16, device="cuda")
        for f in (lib.attn_rope_axes, lib.attn_rope_axes_bwd):
            with pytest.raises(lib.AttnError):
                f(q, None, *rest, q_out=one.expand(2, 3, 5, 64))
            with pytest.raises(lib.AttnError):
                f(q, q, *rest, k_out=one.expand(2, 3, 5, 64))
            with pytest.raises(lib.AttnError):
                f(one.expand(2, 3, 5, 64), None, *rest, q_out=one.expand(2, 3, 5, 64))
        f(one.expand(2, 3, 5, 64), None, *rest)  # (an expanded input is fine)
    both = torch.zeros_like(q)
    with pytest.raises(lib.AttnError):
        lib.attn_rope_axes(q, q, *rest, q_out=both, k_out=both)
