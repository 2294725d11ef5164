"""The further operators in flight at once on two streams, each with tensors and workspaces of its own, give
what they give alone; and a whole decode step (append, decode) captured in two graphs replays on two streams."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def rnd(seed, *s):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def jobs(lib, seed):
    """Callables of one user's calls; the sizes mix both tile shapes of the prefill kernel."""
    q, k, v, g = rnd(seed, 1, 4, 700, 128), rnd(seed + 1, 1, 2, 700, 128), rnd(seed + 2, 1, 2, 700, 128), rnd(seed + 3, 1, 4, 700, 128)
    o, lse = lib.attn_fwd_scoremod(q, k, v, True, softcap=20.0)
    p = rnd(seed + 4, 60, 4, 16, 64)
    table = torch.randperm(60, device="cuda").to(torch.int32).view(6, 10)
    table[1:3, :4] = table[0, :4]
    table[4:, :4] = table[3, :4]
    ctx, shared = i32([100, 130, 159, 64, 70, 160]), i32([4, 4])
    dq, slopes = rnd(seed + 5, 6, 8, 64), torch.rand(8, device="cuda")
    return [lambda: lib.attn_fwd_scoremod(q, k, v, True, softcap=20.0),
            lambda: lib.attn_bwd_scoremod(q, k, v, o, lse, g, True, softcap=20.0),
            lambda: lib.paged_attn_decode_shared(dq, p, p, table, ctx, shared, 3),
            lambda: lib.paged_attn_decode_scoremod(dq, p, p, table, ctx, softcap=20.0, alibi_slopes=slopes)]


def test_two_streams(lib):
    users = [jobs(lib, 10), jobs(lib, 50)]
    want = [[f() for f in u] for u in users]
    streams = [torch.cuda.Stream() for _ in users]
    torch.cuda.synchronize()
    got = []
    for turn in range(10):
        for i in range(4):
            for u, s in zip(range(2), streams):
                with torch.cuda.stream(s):
                    got.append((u, (i + turn) % 4, users[u][(i + turn) % 4]()))
    torch.cuda.synchronize()
    assert lib.attn_check_device_status() == 0
    for u, i, r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[u][i])), (u, i)


def test_two_graphs_of_a_decode_step(lib):
    def step(seed):
        B, H, Hkv, d = 4, 8, 2, 128
        kp, vp = rnd(seed, 40, Hkv, 16, d), rnd(seed + 1, 40, Hkv, 16, d)
        table = torch.randperm(40, device="cuda").to(torch.int32).view(4, 10)
        new = rnd(seed + 2, B, 1, H + 2 * Hkv, d).transpose(1, 2)
        cs = torch.rand(160, d, device="cuda")
        start = i32([20, 63, 0, 140])

        def run():
            q = lib.paged_kv_append_rope(new[:, :H], new[:, H:H + Hkv], new[:, H + Hkv:], kp, vp, cs, table, start)
            return lib.paged_attn_decode_scoremod(q.view(B, H, d), kp, vp, table, start + 1, softcap=30.0)
        return run
    runs = [step(100), step(200)]
    want = [r() for r in runs]
    graphs, outs = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert lib.attn_check_device_status() == 0
