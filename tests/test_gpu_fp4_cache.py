"""Append into the 4-bit cache, and its pages as bf16, against the format's definition (fp4_ref).

Without a rotation every step is one fp32 operation, correctly rounded: codes and scales agree bit for bit.  With one, a
rotated value is off by at most 2^-22 (|x| + |y|) in fp32, so it may fall on the other side of a border: the scale is then
a neighbour (2^-3 of itself away), and a value is within half a step of its size plus that of the definition's."""
import pytest
import torch

import fp4_ref as F
from test_gpu_append_rope import angles, rotate64

pytestmark = pytest.mark.gpu
KS, VS = 0.0113, 0.37


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


def make(B, H, Hkv, N, d, start, W, seed, fused=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    qkv = rnd(B, N, H + 2 * Hkv, d)
    qkv[..., :16] *= 2.0 ** -30  # a block whose scale rounds to zero
    if N > 2:
        qkv[:, 1] *= 2.0 ** 40   # a token past the largest scale
    qkv = qkv.cuda().transpose(1, 2)
    x = [qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]]
    if not fused:
        x = [t.contiguous() for t in x]
    n = B * W
    table = torch.randperm(n, generator=g).view(B, W).to(torch.int32)
    pools = [torch.randint(0, 256, (n + 1, Hkv, 9 * d), generator=g, dtype=torch.uint8) for _ in range(2)]
    return dict(q=x[0], k=x[1], v=x[2], table=table, pools=pools, start=start)


def append(lib, x, **kw):
    kp, vp = (p.cuda() for p in x["pools"])
    kw.setdefault("q", None)
    q = kw.pop("q")
    r = lib.paged_kv_append_fp4(q, x["k"], x["v"], kp, vp, KS, VS, x["table"].cuda(),
                                torch.tensor(x["start"], dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    return r, kp.cpu(), vp.cpu()


def places_of(x, N, new=None, max_pos=1 << 40):
    """(b, t, page, slot) of the tokens that land in a page."""
    W, P = x["table"].shape[1], x["pools"][0].shape[0]
    for b, start in enumerate(x["start"]):
        start = max(start, 0)
        for t in range(N if new is None else min(max(new[b], 0), N)):
            pos = start + t
            if pos < max_pos and pos // 16 < W and 0 <= int(x["table"][b, pos // 16]) < P:
                yield b, t, int(x["table"][b, pos // 16]), pos % 16


CASES = [(1, 1, 1, 32, [0]), (3, 12, 1, 64, [0, 15, 31]), (2, 1, 5, 80, [14, 31]), (2, 2, 37, 96, [0, 17]), (3, 8, 1, 128, [17, 0, 5]),
         (2, 2, 130, 128, [3, 50]), (1, 3, 33, 64, [9])]  # B, Hkv, N, d, start


@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}kv{c[1]}N{c[2]}d{c[3]}" for c in CASES])
@pytest.mark.parametrize("fused", [True, False], ids=["views", "dense"])
def test_without_rotation_bit_for_bit(lib, case, fused):
    B, Hkv, N, d, start = case
    x = make(B, 2, Hkv, N, d, start, (max(start) + N + 15) // 16, 3, fused)
    want = [p.clone() for p in x["pools"]]
    for b, t, page, slot in places_of(x, N):
        F.write(want[0], page, slot, *F.quantise(x["k"][b, :, t].cpu(), KS), False)
        F.write(want[1], page, slot, *F.quantise(x["v"][b, :, t].cpu(), VS), True)
    r, kp, vp = append(lib, x)
    assert r is None and torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_padding_unmapped_pages_and_ends(lib):
    # nothing new; part; past the table's capacity; a negative start; more than Nnew; the largest int
    start, new = [5, 40, 60, -3, 1, 2**31 - 1], [0, 9, 21, 21, 1000, 3]
    x = make(6, 2, 2, 21, 64, start, 4, 6)
    x["table"][1, 2], x["table"][3, 0] = -1, x["pools"][0].shape[0]
    want = [p.clone() for p in x["pools"]]
    for b, t, page, slot in places_of(x, 21, new):
        F.write(want[0], page, slot, *F.quantise(x["k"][b, :, t].cpu(), KS), False)
        F.write(want[1], page, slot, *F.quantise(x["v"][b, :, t].cpu(), VS), True)
    _, kp, vp = append(lib, x, new_lens=torch.tensor(new, dtype=torch.int32).cuda())
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def near(got, want64, slack, scale):
    """The stored values of a token, [Hkv, d] in units of the tensor's scale, against the exact ones: within half a step of a
    code under the block's exact scale, that scale's own rounding (half a step, 2^-4 of it or 2^-10, moves a value by at most
    6 times that through its code's range) and fp32's."""
    u = want64 / scale
    m = u.unflatten(-1, (-1, 16)).abs().amax(-1).repeat_interleave(16, -1)
    s = (m / 6).clamp(max=448.0)
    s_off = torch.maximum(s * 2.0 ** -4, torch.full_like(s, 2.0 ** -10))
    hi = (s + s_off) * 1.0001
    r = u.abs() / hi
    # past the range of the scale only the sign and the largest value are left
    step = torch.where(r <= 2, 0.25, torch.where(r <= 4, 0.5, 1.0)) * hi
    tol = torch.where(s < 448, step + 6 * s_off * 2 + slack / scale, u.abs() + 6 * 448)
    assert ((got - u).abs() <= tol * 1.0001 + 1e-30).all(), float(((got - u).abs() / tol).max())


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("axes", [0, 3], ids=["places", "axes"])
@pytest.mark.parametrize("d, r", [(32, 16), (64, 64), (80, 80), (96, 48), (128, 128)])
def test_with_rotation(lib, d, r, axes, inter):
    B, H, Hkv, N, start = 3, 5, 2, 19, [0, 13, 7]
    x = make(B, H, Hkv, N, d, start, 3, 8)
    g = torch.Generator().manual_seed(9)
    cs = angles(64, r)
    pos = torch.randint(0, 64, (3, B, N), generator=g)
    pos[1, 1, 4] = 64 if axes else 0   # outside the table: padding
    pos[0, 2, 18] = -1 if axes else 0
    pair = bytes(torch.randint(0, 3, (r // 2,), generator=g).tolist())
    kw = dict(positions=pos.int().cuda(), pair_axis=pair) if axes else {}
    before = [p.clone() for p in x["pools"]]
    q_out = torch.full((B, H, N, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out, kp, vp = append(lib, x, q=x["q"], cos_sin=cs.cuda(), interleaved=inter, q_out=q_out, **kw)
    assert out is q_out
    got = [F.read(kp, False), F.read(vp, True)]
    touched = torch.zeros(kp.shape[0], 16, dtype=torch.bool)
    col = torch.arange(r // 2)
    for b in range(B):
        for t in range(N):
            if axes:
                ok = bool(((pos[:, b, t] >= 0) & (pos[:, b, t] < 64)).all())
                row = pos[torch.tensor(list(pair)), b, t].clamp(0, 63)
            else:
                ok, row = True, torch.full((r // 2,), start[b] + t)
            if not ok:
                assert (q_out[b, :, t] == 7).all()
                continue
            z = torch.cat([cs[row, col], cs[row, r // 2 + col]]).double()[None]
            wq, sq = rotate64(x["q"][b, :, t:t + 1].cpu().double(), z, inter)
            assert ((q_out[b, :, t:t + 1].cpu().double() - wq).abs() <= 2.0 ** -8 * wq.abs() + sq).all()
            wk, sk = rotate64(x["k"][b, :, t:t + 1].cpu().double(), z, inter)
            page, slot = int(x["table"][b, (start[b] + t) // 16]), (start[b] + t) % 16
            touched[page, slot] = True
            near(got[0][page, :, slot], wk[:, 0], sk[:, 0], KS)
            cv, sv = F.quantise(x["v"][b, :, t].cpu(), VS)
            one = before[1][:1].clone()
            F.write(one, 0, slot, cv, sv, True)
            assert torch.equal(F.read(one, True)[0, :, slot], got[1][page, :, slot])
    for p, old, value in ((kp, before[0], False), (vp, before[1], True)):
        same = (F.read(p, value) == F.read(old, value)) | F.read(old, value).isnan()
        assert same.transpose(1, 2)[~touched].all()
    again = torch.full_like(q_out, 7.0)
    x["pools"] = [kp, vp]
    _, kp2, vp2 = append(lib, x, q=x["q"], cos_sin=cs.cuda(), interleaved=inter, q_out=again, **kw)
    assert torch.equal(again, q_out) and torch.equal(kp2, kp) and torch.equal(vp2, vp)  # the same tokens again
    x["pools"] = before
    _, kp3, vp3 = append(lib, x, q=None, cos_sin=cs.cuda(), interleaved=inter, **kw)
    assert torch.equal(kp3, kp) and torch.equal(vp3, vp)


@pytest.mark.parametrize("d", [32, 64, 80, 96, 128])
def test_unpack_bit_for_bit(lib, d):
    P, Hkv = 7, 3
    g = torch.Generator().manual_seed(d)
    pools = [torch.randint(0, 256, (P, Hkv, 9 * d), generator=g, dtype=torch.uint8) for _ in range(2)]
    for p in pools:
        p[..., 8 * d:] &= 0x7E  # no NaN among the scales
    ids = torch.tensor([3, -1, 0, P, 6, 3], dtype=torch.int32)
    out = [torch.full((6, Hkv, 16, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    r = lib.paged_kv_unpack_fp4(pools[0].cuda(), pools[1].cuda(), KS, VS, ids.cuda(), k_out=out[0], v_out=out[1])
    assert r[0] is out[0] and r[1] is out[1]
    for o, p, s, value in ((out[0], pools[0], KS, False), (out[1], pools[1], VS, True)):
        want = (F.read(p, value).float() * torch.tensor(s, dtype=torch.float32)).to(torch.bfloat16)
        for i, page in enumerate(ids.tolist()):
            assert torch.equal(o[i].cpu(), want[page] if 0 <= page < P else torch.full_like(want[0], 5.0)), i
    one = lib.paged_kv_unpack_fp4(pools[0].cuda(), pools[1].cuda(), KS, VS, ids[:1].cuda())
    assert torch.equal(one[0][0], out[0][0]) and one[1].shape == (1, Hkv, 16, d)


def test_pool_past_32_bit_offsets(lib):
    Hkv, d = 8, 128
    pages = (1 << 32) // (Hkv * 9 * d) + 64
    kp = torch.zeros(pages, Hkv, 9 * d, dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    k = torch.randn(1, Hkv, 20, d, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16).cuda()
    table, start = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda"), torch.tensor([7], dtype=torch.int32).cuda()
    lib.paged_kv_append_fp4(None, k, k, kp, vp, KS, VS, table, start)
    small = [torch.zeros(4, Hkv, 9 * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    near_table = torch.tensor([[3, 1]], dtype=torch.int32, device="cuda")
    lib.paged_kv_append_fp4(None, k, k, *small, KS, VS, near_table, start)
    assert torch.equal(kp[-4:], small[0]) and torch.equal(vp[-4:], small[1]) and int(kp[:-4].max()) == 0
    a = lib.paged_kv_unpack_fp4(kp, vp, KS, VS, table[0])
    b = lib.paged_kv_unpack_fp4(*small, KS, VS, near_table[0])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q, ctx = torch.randn(1, 16, d).to(torch.bfloat16).cuda(), torch.tensor([27], dtype=torch.int32).cuda()
    x, y = lib.paged_attn_decode_fp4(q, kp, vp, KS, VS, table, ctx), lib.paged_attn_decode_fp4(q, *small, KS, VS, near_table, ctx)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_other_stream_and_captured_graph(lib):
    x = make(4, 8, 2, 1, 128, [0, 5, 15, 33], 4, 9)
    cs = angles(64, 128).cuda()
    call = lambda kp, vp, start, **kw: lib.paged_kv_append_fp4(  # noqa: E731
        x["q"], x["k"], x["v"], kp, vp, KS, VS, x["table"].cuda(), start, cos_sin=cs, **kw)
    a, b = [p.cuda() for p in x["pools"]], [p.cuda() for p in x["pools"]]
    start, table = torch.tensor(x["start"], dtype=torch.int32).cuda(), x["table"].cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q_out = lib.paged_kv_append_fp4(x["q"], x["k"], x["v"], *a, KS, VS, table, start, cos_sin=cs, stream=side)
    side.synchronize()
    assert torch.equal(call(*b, start), q_out) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ids = table.flatten()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.paged_kv_append_fp4(x["q"], x["k"], x["v"], *a, KS, VS, table, start, cos_sin=cs, q_out=q_out)
        bits = lib.paged_kv_unpack_fp4(*a, KS, VS, ids)
    for _ in range(3):
        graph.replay()
        want = call(*b, start)
        assert torch.equal(want, q_out) and torch.equal(a[1], b[1])
        assert torch.equal(bits[1].view(torch.int16), lib.paged_kv_unpack_fp4(*b, KS, VS, ids)[1].view(torch.int16))
        start.add_(1)
