"""The compiled argument marshalling and the one in Python give the same results and the same errors."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    binding._torch()
    if binding._fast is None:
        pytest.skip("the compiled marshalling was not built here")
    return binding


def rnd(*s):
    return torch.randn(*s, device="cuda").to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    """name -> (function, positional arguments, optional arguments with the values a caller may pass)."""
    torch.manual_seed(0)
    q, k, v, g = rnd(2, 4, 40, 64), rnd(2, 2, 40, 64), rnd(2, 2, 40, 64), rnd(2, 4, 40, 64)
    o, lse = rnd(2, 4, 40, 64), torch.randn(2, 4, 40, device="cuda").abs() + 5
    pages, codes = rnd(8, 2, 16, 64), torch.randint(0, 100, (8, 2, 16, 64), dtype=torch.uint8, device="cuda")
    table, ctx, dq = i32([[0, 1, 2], [3, 4, 5]]), i32([40, 17]), rnd(2, 4, 64)
    slopes = torch.rand(4, device="cuda")
    cs = torch.rand(64, 64, device="cuda")
    mod = dict(softcap=30.0, alibi_slopes=slopes, key_begin=i32([[0] * 40] * 2), key_end=i32([[40] * 40] * 2), kv_lens=i32([40, 33]))
    new = rnd(2, 3, 8, 64).transpose(1, 2)
    return {
        "attn_fwd_scoremod": ((q, k, v, True), dict(scale=0.1, **mod)),
        "attn_bwd_scoremod": ((q, k, v, o, lse, g, False), dict(scale=0.1, **mod)),
        "paged_attn_decode_scoremod": ((dq, pages, pages, table, ctx), dict(scale=0.2, softcap=20.0, alibi_slopes=slopes, key_begin=i32([3, 0]))),
        "paged_attn_decode_scoremod_fp8": ((dq, codes, codes, 0.02, 0.03, table, ctx), dict(softcap=20.0)),
        "paged_attn_decode_shared": ((dq, pages, pages, table, ctx, i32([1]), 2), dict(scale=0.2)),
        "paged_attn_decode_shared_fp8": ((dq, codes, codes, 0.02, 0.03, table, ctx, i32([1, 0]), 1), {}),
        "paged_kv_append_rope": ((new[:, :4], new[:, 4:6], new[:, 6:], pages, pages.clone(), cs, table, i32([0, 9])), dict(interleaved=True, new_lens=i32([3, 2]))),
        "paged_kv_append_rope_fp8": ((new[:, :4], new[:, 4:6], new[:, 6:], codes, codes.clone(), 0.02, 0.03, cs, table, i32([0, 9])), {}),
    }


NAMES = ["attn_fwd_scoremod", "attn_bwd_scoremod", "paged_attn_decode_scoremod",
         "paged_attn_decode_scoremod_fp8", "paged_attn_decode_shared", "paged_attn_decode_shared_fp8",
         "paged_kv_append_rope", "paged_kv_append_rope_fp8"]


def outcome(f, args, kw):
    try:
        r = f(*args, **kw)
    except Exception as e:
        return type(e).__name__, str(e)
    torch.cuda.synchronize()
    r = r if isinstance(r, tuple) else (r,)
    # (the rows of padding of an allocated q_out are uninitialised: compare what was written elsewhere)
    return tuple(None if t is None else t.clone() for t in r)


def both(lib, monkeypatch, name, args, kw):
    fast = outcome(getattr(lib, name), args, kw)
    with monkeypatch.context() as m:
        m.setattr(lib, "_fast", None)
        slow = outcome(getattr(lib, name), args, kw)
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert (a == b) if not isinstance(a, torch.Tensor) else torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (name, a, b)
    return fast


@pytest.mark.parametrize("name", NAMES)
def test_same_results(lib, monkeypatch, name):
    args, kw = calls()[name]
    if name.startswith("paged_kv"):
        kw = dict(kw, q_out=torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda"))
    both(lib, monkeypatch, name, args, kw)
    both(lib, monkeypatch, name, args, {k: v for k, v in kw.items() if k in ("q_out", "interleaved")})  # all defaults
    if name.startswith("paged_attn") or name == "attn_fwd_scoremod":
        assert both(lib, monkeypatch, name, args, dict(kw, return_lse=False))[1] is None
    if name.startswith("paged_kv"):
        both(lib, monkeypatch, name, (None, *args[1:]), {k: v for k, v in kw.items() if k != "q_out"})


@pytest.mark.parametrize("name", NAMES)
def test_outputs_given_are_the_ones_returned(lib, name):
    args, kw = calls()[name]
    if name.startswith("paged_kv"):
        out = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
        assert getattr(lib, name)(*args, **dict(kw, q_out=out)) is out
    elif name == "attn_bwd_scoremod":
        g = [torch.empty_like(t) for t in args[:3]]
        r = lib.attn_bwd_scoremod(*args, **dict(kw, dq=g[0], dk=g[1], dv=g[2]))
        assert all(x is y for x, y in zip(r, g))
    else:
        out, lse = torch.empty_like(args[0]), torch.empty(args[0].shape[:-1], device="cuda")
        r = getattr(lib, name)(*args, **dict(kw, out=out, lse=lse))
        assert r[0] is out and r[1] is lse


@pytest.mark.parametrize("name", NAMES)
def test_same_errors(lib, monkeypatch, name):
    args, kw = calls()[name]
    for i, a in enumerate(args):
        if isinstance(a, torch.Tensor):
            for bad in (a.cpu(), a.double() if a.is_floating_point() else a.float(), a[:0], a[None], None, 3):
                if name.startswith("paged_kv") and i == 0 and bad is None:
                    continue  # no query: allowed
                r = both(lib, monkeypatch, name, (*args[:i], bad, *args[i + 1:]), kw)
                assert isinstance(r[0], str), (name, i)
    for k, a in kw.items():
        if isinstance(a, torch.Tensor):
            for bad in (a.cpu(), a.double(), a[:1], a[None]):
                assert isinstance(both(lib, monkeypatch, name, args, dict(kw, **{k: bad}))[0], str), (name, k)
    extra = {"attn_bwd_scoremod": dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
             "attn_fwd_scoremod": dict(softcap=-1.0)}
    if name.startswith("paged_attn"):
        extra[name] = dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    if name in extra:
        assert both(lib, monkeypatch, name, args, dict(kw, **extra[name]))[0] == "AttnError"
    if "scoremod" in name:
        for cap in (-1.0, float("nan"), float("inf"), 1e31):
            assert both(lib, monkeypatch, name, args, dict(kw, softcap=cap))[0] == "AttnError"


def test_no_memory(lib, monkeypatch):
    q, pages = rnd(64, 32, 128), rnd(1, 8, 16, 128)
    table, ctx = torch.zeros(64, 4096, dtype=torch.int32, device="cuda"), i32([16] * 64)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    room = torch.cuda.memory_reserved() + (32 << 20)  # the workspace takes 69 MB
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    try:
        for fast in (lib._fast, None):
            with monkeypatch.context() as m:
                m.setattr(lib, "_fast", fast)
                with pytest.raises(torch.OutOfMemoryError):
                    lib.paged_attn_decode_scoremod(q, pages, pages, table, ctx)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.isfinite(lib.paged_attn_decode_scoremod(q, pages, pages, table, ctx)[0]).all()


def test_a_stream_of_its_own_takes_the_same_path_to_the_result(lib):
    args, kw = calls()["paged_attn_decode_scoremod"]
    want = lib.paged_attn_decode_scoremod(*args, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        here = lib.paged_attn_decode_scoremod(*args, **kw)  # the compiled path on the current side stream
    given = lib.paged_attn_decode_scoremod(*args, stream=side, **kw)
    side.synchronize()
    for r in (here, given):
        assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])
