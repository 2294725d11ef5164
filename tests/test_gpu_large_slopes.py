"""The distance bias over the whole range of its slopes, which may be any finite number, against 64 bits.

A score x - slope distance is two roundings of the bias and one of the sum: off by at most 3 * 2^-24 of the bias
and 2^-24 of the score, and the conversions to the log2 domain and back add as much again.  Where a row sees its
own position, every key whose weight counts (bias within 20 of the smallest one's, weights below 2e-9 else) has a
bias of at most 20, so LSE and weights move by at most 20 * 2^-21 = 1e-5, within the bounds of the other tests
(LSE 1e-4, weights 4e-4).  Where it does not, LSE is off by 2^-21 of itself more, and a row's weights by 2^-21 of
the bias: those rows are checked with slopes that keep that below 1e-4, or whose largest weight is all of the sum."""
import pytest
import torch

from scoremod_ref import backward, forward
from test_gpu_scoremod import grad_bounds, o_bound, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


SLOPES = [0.25, 3.0, -0.01, 100.0, 1e4, 1e8, 1e20, 3e38]


def inputs(N, d, Hkv=4):
    H = len(SLOPES)
    return rand(1, 1, H, N, d), rand(2, 1, Hkv, N, d), rand(3, 1, Hkv, N, d), rand(4, 1, H, N, d), torch.tensor(SLOPES)


@pytest.mark.parametrize("cap", [0.0, 20.0], ids=["bias", "cap_bias"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both_ways"])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_and_backward(lib, d, causal, cap):
    q, k, v, g, sl = inputs(300, d)
    scale = d ** -0.5
    c = [t.cuda() for t in (q, k, v)]
    o, lse = lib.attn_fwd_scoremod(*c, causal, scale, softcap=cap, alibi_slopes=sl.cuda())
    want, wl, w, t = forward(q, k, v, causal, scale, cap, sl)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert (lse.cpu().double() - wl).abs().max() <= 1e-4, (lse.cpu().double() - wl).abs().amax((0, 2))
    assert ((o.cpu().double() - want).abs() <= o_bound(w, v, want)).all()
    got = lib.attn_bwd_scoremod(*c, o, lse, g.cuda(), causal, scale, softcap=cap, alibi_slopes=sl.cuda())
    ref = backward(q, k, v, g, causal, scale, cap, sl)
    for name, x, y, tol in zip(("dq", "dk", "dv"), got, ref, grad_bounds(q, k, v, g, want, w, t, scale, ref)):
        assert torch.isfinite(x).all(), name
        err = (x.cpu().double() - y).abs()
        assert (err <= tol).all(), (name, float((err / tol).max()))


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_do_not_see_their_own_position(lib, d):
    q, k, v, _, sl = inputs(400, d)
    end = (torch.arange(400) - 40).clamp(min=0).expand(1, 400).contiguous().to(torch.int32)
    keep = [0, 1, 2, 3, 4, 5]  # with 1e20 and 3e38 the scores approach and leave fp32's range
    o, lse = lib.attn_fwd_scoremod(q.cuda(), k.cuda(), v.cuda(), False, d ** -0.5, alibi_slopes=sl.cuda(), key_end=end.cuda())
    want, wl, w, _ = forward(q, k, v, False, d ** -0.5, 0.0, sl, None, end)
    assert not torch.isnan(o).any() and not torch.isnan(lse).any()
    got = lse.cpu().double()[:, keep]
    assert torch.equal(torch.isneginf(got), torch.isneginf(wl[:, keep]))
    err = (got - wl[:, keep]).nan_to_num(0.0).abs()
    assert (err <= 1e-4 + 2.0 ** -21 * wl[:, keep].abs().nan_to_num(0.0, 0.0, 0.0)).all()
    assert ((o.cpu().double() - want).abs() <= o_bound(w, v, want))[:, keep].all()


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-20])
def test_slopes_beside_the_smallest_scales(lib, scale):
    # the slope divided by the scale leaves fp32's range
    q, k, v, _, sl = inputs(200, 64)
    o, lse = lib.attn_fwd_scoremod(q.cuda(), k.cuda(), v.cuda(), True, scale, alibi_slopes=sl.cuda())
    want, wl, w, _ = forward(q, k, v, True, scale, 0.0, sl)
    assert (lse.cpu().double() - wl).abs().max() <= 1e-4
    assert ((o.cpu().double() - want).abs() <= o_bound(w, v, want)).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_decode(lib, fp8):
    import paged_ref as R
    from test_gpu_decode_scoremod import make, run
    ctx = [300, 17, 1]
    x = make(3, len(SLOPES), 4, 64, ctx, fp8, 3)
    got = run(lib, x, fp8, alibi_slopes=torch.tensor(SLOPES))
    R.check(got[0].cpu(), got[1].cpu(), *R.decode(x[0], x[1], x[2], x[3], ctx, 64 ** -0.5, fp8, 0.0, torch.tensor(SLOPES)))
