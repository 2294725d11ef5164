"""The compiled argument marshalling of the 4-bit cache, the rotation by several axes and the pages' calls gives the results
and the errors of the one in Python, on given and on allocated outputs, and on a stream of its own."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


PAIR = bytes([0] * 16 + [1] * 16)
S = (0.02, 0.03)


def calls():
    """name -> (positional arguments, optional arguments, outputs a caller may give); fresh tensors at each call."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    four = [torch.randint(0, 0x70, (8, 2, 9 * 64), generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    new, dq = rnd(2, 3, 8, 64).transpose(1, 2), rnd(2, 4, 64)
    table, ctx, start = i32([[0, 1, 2], [3, 4, 5]]), i32([40, 17]), i32([0, 9])
    cs, pos = torch.rand(64, 64, generator=g, device="cuda"), i32([[[1, 2, 3], [4, 5, 6]], [[9, 8, 7], [3, 2, 1]]])
    heads = (new[:, :4], new[:, 4:6], new[:, 6:])
    bf, codes = [rnd(8, 2, 16, 64) for _ in range(2)], [torch.randint(0, 100, (8, 2, 16, 64), generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    zeros = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    more = dict(interleaved=True, new_lens=i32([3, 2]), q_out=zeros(2, 4, 3, 64))
    z32 = lambda *s: zeros(*s, t=torch.int32)  # noqa: E731
    tree, ref = i32([[0, 1, -1], [0, 2, 3]]), i32([2, 1, 1, 1, 0, 0, 0, 0])
    return {
        "paged_attn_decode_fp4": ((dq, *four, *S, table, ctx), dict(scale=0.2, softcap=20.0, alibi_slopes=torch.rand(4, device="cuda", generator=g), key_begin=i32([3, 0])),
                                  dict(out=zeros(2, 4, 64), lse=zeros(2, 4, t=torch.float32))),
        "paged_kv_append_fp4": ((*heads, *four, *S, table, start), dict(cos_sin=cs, positions=pos, pair_axis=PAIR, **more), {}),
        "paged_kv_append_rope_axes": ((*heads, *bf, cs, pos, PAIR, table, start), more, {}),
        "paged_kv_append_rope_axes_fp8": ((*heads, *codes, *S, cs, pos, PAIR, table, start), more, {}),
        "paged_kv_unpack_fp4": ((*four, *S, i32([3, 0, 7])), {}, dict(k_out=zeros(3, 2, 16, 64), v_out=zeros(3, 2, 16, 64))),
        "attn_rope_axes": ((*heads[:2], cs, pos, PAIR), dict(interleaved=True), dict(q_out=zeros(2, 4, 3, 64), k_out=zeros(2, 2, 3, 64))),
        "attn_rope_axes_bwd": ((*heads[:2], cs, pos[:, :1].contiguous(), PAIR), {}, dict(q_out=zeros(2, 4, 3, 64), k_out=zeros(2, 2, 3, 64))),
        "paged_kv_fork": ((tree, i32([20, 40]), i32([1, 1, 0, -1]), ref), {}, dict(page_table_out=z32(4, 3), ctx_lens_out=z32(4), ref_counts_out=z32(8))),
        "paged_kv_reserve": ((tree, i32([20, 40]), i32([1, 8]), ref), {},
                             dict(page_table_out=z32(2, 3), ref_counts_out=z32(8), reserved=z32(2), src_pages=z32(2), dst_pages=z32(2))),
        "paged_kv_compact": ((i32([[7, 2, -1], [7, 5, -1]]), i32([0, 0, 1, 0, 0, 1, 0, 2])), {},
                             dict(page_table_out=z32(2, 3), ref_counts_out=z32(8), src_pages=z32(8), dst_pages=z32(8), count=z32(1))),
        "paged_kv_copy_pages": ((bf, i32([1, 2]), i32([5, 6])), dict(count=i32([1])), {}),
    }


NAMES = sorted(calls()) if torch.cuda.is_available() else ["-"]


def tensors(x):
    if isinstance(x, torch.Tensor):
        yield x
    elif isinstance(x, (list, tuple)):
        for y in x:
            yield from tensors(y)
    elif isinstance(x, dict):
        yield from tensors(list(x.values()))


def outcome(lib, name, args, kw):
    """What a call returns and leaves in its arguments, or its error."""
    try:
        r = getattr(lib, name)(*args, **kw)
    except Exception as e:
        return type(e).__name__, str(e)
    torch.cuda.synchronize()
    return [t.clone() for t in tensors([r, args, kw])]


def both(lib, monkeypatch, name, change=lambda a, k: (a, k)):
    got = []
    for fast in (True, False):
        args, kw, _ = calls()[name]
        args, kw = change(list(args), dict(kw))
        with monkeypatch.context() as m:
            if not fast:
                m.setattr(lib, "_fast", None)
            got.append(outcome(lib, name, args, kw))
    a, b = got
    if isinstance(a, tuple) or isinstance(b, tuple):
        assert a == b, (name, a, b)
    else:
        assert len(a) == len(b) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b)), name
    return a


@pytest.mark.parametrize("name", NAMES)
def test_same_results(lib, monkeypatch, name):
    assert not isinstance(both(lib, monkeypatch, name), tuple)
    keep = ("q_out", "interleaved", "cos_sin")  # all other options left out
    assert not isinstance(both(lib, monkeypatch, name, lambda a, k: (a, {n: v for n, v in k.items() if n in keep})), tuple)
    if name == "paged_attn_decode_fp4":
        assert not isinstance(both(lib, monkeypatch, name, lambda a, k: (a, dict(k, return_lse=False))), tuple)
    if "append" in name:
        assert not isinstance(both(lib, monkeypatch, name, lambda a, k: ([None] + a[1:], {n: v for n, v in k.items() if n != "q_out"})), tuple)
    if "append" in name or "rope" in name:  # the axes as a list: converted
        def listed(a, k):
            a = [list(x) if isinstance(x, bytes) else x for x in a]
            return a, {n: list(v) if isinstance(v, bytes) else v for n, v in k.items()}
        assert not isinstance(both(lib, monkeypatch, name, listed), tuple)
    if name.startswith("attn_rope"):
        assert not isinstance(both(lib, monkeypatch, name, lambda a, k: ([a[0], None] + a[2:], k)), tuple)
    if name == "paged_kv_append_fp4":
        assert not isinstance(both(lib, monkeypatch, name, lambda a, k: ([None] + a[1:], dict(new_lens=k["new_lens"]))), tuple)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_given_are_the_ones_returned(lib, monkeypatch, name):
    for fast in (lib._fast, None):
        with monkeypatch.context() as m:
            m.setattr(lib, "_fast", fast)
            args, kw, outs = calls()[name]
            want = getattr(lib, name)(*args, **kw)
            args, kw, outs = calls()[name]
            got = getattr(lib, name)(*args, **kw, **outs)
            if outs:
                assert all(x is y for x, y in zip(got, outs.values()))
                assert all(torch.equal(x, y) for x, y in zip(got, want))
            elif "q_out" in kw:
                assert got is kw["q_out"]


@pytest.mark.parametrize("name", NAMES)
def test_same_errors(lib, monkeypatch, name):
    args, kw, outs = calls()[name]
    kw = dict(kw, **outs)
    for i, a in enumerate(args):
        for bad in (lambda x: x.cpu(), lambda x: x.double() if x.is_floating_point() else x.float(), lambda x: x[:0], lambda x: x[None],
                    lambda x: None, lambda x: 3):
            def change(al, k, i=i, bad=bad):
                if isinstance(al[i], torch.Tensor):
                    al[i] = bad(al[i])
                elif isinstance(al[i], bytes):
                    al[i] = [7, "x"] if bad(torch.zeros(1)) is None else al[i][:-1]
                return al, k
            if isinstance(a, (torch.Tensor, bytes)):
                none_is_fine = bad(torch.zeros(2)) is None and ((i == 0 and "append" in name) or (i == 1 and "attn_rope" in name))
                r = both(lib, monkeypatch, name, change)
                assert none_is_fine or isinstance(r, tuple), (name, i)
    for n, a in kw.items():
        if isinstance(a, torch.Tensor):
            for bad in (lambda x: x.cpu(), lambda x: x.double(), lambda x: x[None], lambda x: torch.cat([x, x])):
                if n in ("cos_sin", "positions") and bad(a).shape[0] == 2 * a.shape[0]:
                    continue  # a table of more rows, positions with more axes
                r = both(lib, monkeypatch, name, lambda al, k, n=n, bad=bad: (al, dict(k, **{n: bad(kw[n])})))
                assert isinstance(r, tuple), (name, n)
    extra = {"paged_attn_decode_fp4": dict(softcap=-1.0), "paged_kv_reserve": dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
             "paged_kv_compact": dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))}
    if name in extra:
        assert both(lib, monkeypatch, name, lambda a, k: (a, dict(k, **extra[name])))[0] == "AttnError"


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_its_own(lib, name):
    args, kw, _ = calls()[name]
    want = outcome(lib, name, args, kw)
    side = torch.cuda.Stream()
    for given in (True, False):
        args, kw, _ = calls()[name]
        torch.cuda.synchronize()
        if given:
            got = outcome(lib, name, args, dict(kw, stream=side))
        else:
            with torch.cuda.stream(side):
                got = outcome(lib, name, args, kw)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, want))


def test_pools_of_another_kind(lib):
    bf = [torch.zeros(4, 8, device="cuda") for _ in range(2)]
    s = i32([0]), i32([1])
    for bad in ([bf[0], bf[1].cpu()], [bf[0], bf[1][:2]], [bf[0], bf[1].double()], [], [bf[0], 3], [bf[0][:, :3]], [bf[0][:0]]):
        with pytest.raises((ValueError, TypeError, lib.AttnError)):
            lib.paged_kv_copy_pages(bad, *s)
    lib.paged_kv_copy_pages(iter(bf), *s)  # any sequence


def test_two_streams_and_two_graphs(lib):
    """Two users' calls in flight at once, each with tensors and workspaces of its own, and two captured steps that replay on
    two streams, give what they give alone."""
    names = [n for n in NAMES if n != "paged_kv_copy_pages"]
    users = [{n: calls()[n] for n in names} for _ in range(2)]
    for n in names:  # another user's other values
        for t in tensors(users[1][n][0]):
            if t.dtype == torch.bfloat16:
                t.neg_()
    step = lambda u: [getattr(lib, n)(*users[u][n][0], **users[u][n][1]) for n in names]  # noqa: E731
    want = [[t.clone() for t in tensors(step(u))] for u in range(2)]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    got = [[], []]
    for turn in range(5):
        for u in range(2):
            with torch.cuda.stream(streams[u]):
                got[u].append(step(u))
    torch.cuda.synchronize()
    for u in range(2):
        for r in got[u]:
            assert all(torch.equal(x, y) for x, y in zip(tensors(r), want[u]))
    for u in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[u], stream=streams[u]):
            outs.append(step(u))
    for t in tensors(outs):
        t.zero_()
    torch.cuda.synchronize()
    for turn in range(5):
        for u in range(2):
            with torch.cuda.stream(streams[u]):
                graphs[u].replay()
    torch.cuda.synchronize()
    for u in range(2):
        assert all(torch.equal(x, y) for x, y in zip(tensors(outs[u]), want[u]))
    assert lib.attn_check_device_status() == 0
