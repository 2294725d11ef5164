"""A query that holds NaN, or an infinity that its scores meet with both signs, gives NaN in its own outputs, and
nothing else changes: it must not pass for a row that sees no key (O = 0, LSE = -inf)."""
import pytest
import torch

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


def compare(got, clean, bad):
    """bad [B, H]: NaN there, and the clean call's bits elsewhere."""
    bad = bad.cuda()
    assert torch.isnan(got[0][bad]).all() and torch.isnan(got[1][bad]).all()
    assert torch.equal(got[0][~bad], clean[0][~bad]) and torch.equal(got[1][~bad], clean[1][~bad])


def spoil(q, rows):
    q, bad = q.clone(), torch.zeros(q.shape[:2], dtype=torch.bool)
    for b, h in rows:
        q[b, h, 5] = float("nan")
        bad[b, h] = True
    return q, bad


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("mod", [dict(), dict(softcap=20.0), dict(slopes=True)], ids=["plain", "cap", "bias"])
@pytest.mark.parametrize("spare", [2, 2100], ids=["cluster", "workspace"])
def test_decode_with_modified_scores(lib, spare, mod, fp8):
    x = list(make(3, 8, 2, 64, [300, 17, 0], fp8, 3, spare=spare))
    kw = dict(softcap=mod.get("softcap", 0.0), alibi_slopes=torch.full((8,), 0.1) if "slopes" in mod else None)
    clean = run(lib, x, fp8, **kw)
    x[0], bad = spoil(x[0], [(0, 1), (1, 6), (2, 3)])
    bad[2, 3] = False  # sequence 2 sees no token: its query does not matter
    compare(run(lib, x, fp8, **kw), clean, bad)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("once", [False, True], ids=["per_sequence", "per_group"])
def test_decode_of_shared_prefixes(lib, once, fp8):
    # sequence 3 lies in the shared pages alone
    x = make_shared(4, 2, 64, 2, [10, 3], [200, 190, 60, 30], fp8, 4, spare=48000 if once else 1)
    clean = run_shared(lib, x, fp8)
    x["q"], bad = spoil(x["q"], [(0, 1), (3, 3)])
    compare(run_shared(lib, x, fp8), clean, bad)


@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(alibi_slopes=True), dict(softcap=20.0, alibi_slopes=True)],
                         ids=["plain", "cap", "bias", "cap_bias"])
@pytest.mark.parametrize("d", [64, 128])
def test_forward(lib, d, kw):
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, h, 300, d, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    kw = {n: torch.full((4,), 0.1, device="cuda") if n == "alibi_slopes" else a for n, a in kw.items()}
    clean = lib.attn_fwd_scoremod(q, k, v, True, **kw)
    bad = torch.zeros(1, 4, 300, dtype=torch.bool)
    q = q.clone()
    for h, i in ((0, 0), (1, 7), (2, 299)):
        q[0, h, i, 3] = float("nan")
        bad[0, h, i] = True
    compare(lib.attn_fwd_scoremod(q, k, v, True, **kw), clean, bad)
