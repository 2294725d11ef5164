"""Queries of very different magnitudes over an e4m3 cache: each query head is rounded to f16 after a power of
two of its own, so a huge head takes nothing from its neighbours (bounds in paged_ref.check)."""
import pytest
import torch

import paged_ref as R
from test_gpu_decode_scoremod import make, run
from test_gpu_decode_shared import make as make_shared, run as run_shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def enlarge(q, heads, by):
    q = q.float()
    q[:, heads] *= by
    return q.to(torch.bfloat16)


def ordinary(got, want, heads):
    """The bounds on the heads that were not enlarged."""
    keep = [h for h in range(got[0].shape[1]) if h not in heads]
    R.check(got[0].cpu()[:, keep], got[1].cpu()[:, keep], *(t[:, keep] for t in want))


SHAPES = [(4, 1, 64, [300, 17], [2]), (8, 1, 128, [90, 700], [0, 7]), (16, 1, 32, [1, 200], [3, 12]), (40, 2, 80, [130], [5, 39]),
          (12, 2, 96, [1500, 48, 33], [11])]


@pytest.mark.parametrize("by", [2.0 ** 16, 2.0 ** 40, 2.0 ** 120], ids=["2^16", "2^40", "2^120"])
@pytest.mark.parametrize("spare", [2, 2100], ids=["cluster", "workspace"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"H{s[0]}kv{s[1]}d{s[2]}" for s in SHAPES])
def test_decode_with_modified_scores(lib, shape, spare, by):
    H, Hkv, d, ctx, huge = shape
    x = list(make(len(ctx), H, Hkv, d, ctx, True, 3, spare=spare))
    x[0] = enlarge(x[0], huge, by)
    # a huge head's scores lie on the cap's flat ends; from 2^40 on, where a sum of products would have to cancel to
    # 1e-9 to leave them, its LSE is checked too (its weights are a choice of signs, all equal)
    got = run(lib, x, True, softcap=20.0)
    want = R.decode(x[0], x[1], x[2], x[3], ctx, d ** -0.5, True, 20.0)
    ordinary(got, want, huge)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
    if by >= 2.0 ** 40:
        assert (got[1].cpu().double() - want[1])[:, huge].abs().max() <= 1e-4
    got = run(lib, x, True)
    ordinary(got, R.decode(x[0], x[1], x[2], x[3], ctx, d ** -0.5, True), huge)


@pytest.mark.parametrize("once", [False, True], ids=["per_sequence", "per_group"])
def test_decode_of_shared_prefixes(lib, once):
    x = make_shared(8, 2, 64, 2, [10, 3], [200, 190, 60, 77], True, 4, spare=48000 if once else 1)
    x["q"] = enlarge(x["q"], [1, 6], 2.0 ** 40)
    got = run_shared(lib, x, True)
    ordinary(got, R.decode(x["q"], x["k"], x["v"], x["full"], x["ctx"].tolist(), 64 ** -0.5, True), [1, 6])


def test_heads_of_one_magnitude_are_untouched(lib):
    # a factor of one changes nothing: the ordinary heads' bits beside a huge one are those beside an ordinary one
    x = list(make(3, 8, 1, 64, [500, 33, 16], True, 6))
    plain = run(lib, x, True, softcap=20.0)
    x[0] = enlarge(x[0], [4], 2.0 ** 30)
    got = run(lib, x, True, softcap=20.0)
    keep = [0, 1, 2, 3, 5, 6, 7]
    assert torch.equal(got[0][:, keep], plain[0][:, keep]) and torch.equal(got[1][:, keep], plain[1][:, keep])
