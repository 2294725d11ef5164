"""The 4-bit cache and the rotation by several axes on the host: the format's reference against itself, and refusals,
which come back as a status before any device work or are raised by the binding."""
import ctypes

import pytest
import torch

import fp4_ref as F

A = 1 << 20  # fake, 16-byte aligned addresses: the checks fail before any use
S = 0.01


@pytest.fixture(scope="module")
def lib():
    from attn_fwd_02_gb300 import binding
    from attn_fwd_02_gb300 import build as buildmod
    buildmod.build()
    return binding.load_library()


@pytest.mark.parametrize("d", [32, 64, 80, 96, 128])
@pytest.mark.parametrize("value", [False, True])
def test_every_code_and_scale_has_a_place_of_its_own(d, value):
    at, shift, sc = F.places(d, value)
    nibbles = (at * 2 + shift // 4).flatten()
    assert nibbles.unique().numel() == 16 * d and int(nibbles.min()) == 0 and int(nibbles.max()) == 16 * d - 1
    assert sc[:, ::16].flatten().unique().numel() == d and int(sc.min()) == 8 * d and int(sc.max()) == 9 * d - 1


def test_reference_quantiser_is_off_by_half_a_step():
    x = torch.randn(3, 5, 64, generator=torch.Generator().manual_seed(1))
    codes, scales = F.quantise(x, S)
    p = torch.zeros(1, 3, 9 * 64, dtype=torch.uint8)
    for t in range(5):
        F.write(p, 0, t, codes[:, t], scales[:, t], True)
    y = F.read(p, True)[0, :, :5] * S
    s = (scales.view(torch.float8_e4m3fn).double() * S).repeat_interleave(16, -1)
    r = x.double().abs() / s
    assert ((y - x.double()).abs() <= s * 1.0001 * torch.where(r <= 2, 0.25, torch.where(r <= 4, 0.5, 1.0))).all()


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


AXES = bytes([0] * 16 + [1] * 16)


def append4(lib, q=A, qs=None, k=A, ks=None, v=A, vs=None, qo=A, kp=A, vp=A, kscale=S, vscale=S, cs=A, rope=64, max_pos=100,
            inter=0, pos=A, axes=2, pair=AXES, table=A, start=A, new=None, ps=16, B=2, H=4, Hkv=2, N=3, d=64, W=8, P=9):
    return lib.paged_kv_append_fp4(q, qs, k, ks, v, vs, qo, kp, vp, kscale, vscale, cs, rope, max_pos, inter, pos, axes, pair,
                                   table, start, new, ps, B, H, Hkv, N, d, W, P, None)


@pytest.mark.parametrize("bad, status", [
    (dict(k=None), 1), (dict(vp=None), 1), (dict(table=None), 1), (dict(q=None), 1), (dict(cs=None), 1),
    (dict(cs=None, pos=None), 1), (dict(cs=None, q=None, qo=None), 1), (dict(kscale=0.0), 1), (dict(vscale=float("nan")), 1),
    (dict(kscale=1e-38), 1), (dict(vscale=float("inf")), 1), (dict(axes=0), 1), (dict(pair=None), 1),
    (dict(pair=bytes([2] * 32)), 1), (dict(B=1 << 20, N=1 << 12), 1), (dict(N=0), 1), (dict(inter=2), 1),
    (dict(axes=5), 2), (dict(rope=72), 2), (dict(rope=80), 2), (dict(d=48, rope=48), 2), (dict(ps=32), 2),
    (dict(pos=A + 2), 3), (dict(kp=A + 8), 3), (dict(start=A + 1), 3), (dict(ks=strides(768, 68, 256)), 3),
    (dict(kp=A + 8, cs=None, pos=None, q=None, qo=None), 3),
])
def test_append_refusals(lib, bad, status):
    assert append4(lib, **bad) == status


def axes_append(lib, fp8, pos=A, axes=2, pair=AXES, rope=64, cs=A, ks=S):
    head = (A, None, A, None, A, None, A, A, A) + ((ks, S) if fp8 else ())
    f = lib.paged_kv_append_rope_axes_fp8 if fp8 else lib.paged_kv_append_rope_axes
    return f(*head, cs, rope, 100, 0, pos, axes, pair, A, A, None, 16, 2, 4, 2, 3, 64, 8, 9, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_axes_append_refusals(lib, fp8):
    assert axes_append(lib, fp8, pos=None) == 1 and axes_append(lib, fp8, pair=None) == 1
    assert axes_append(lib, fp8, axes=0) == 1 and axes_append(lib, fp8, pair=bytes([9] * 32)) == 1
    assert axes_append(lib, fp8, axes=5) == 2 and axes_append(lib, fp8, rope=24) == 2
    assert axes_append(lib, fp8, pos=A + 1) == 3 and axes_append(lib, fp8, cs=None) == 1
    assert not fp8 or axes_append(lib, True, ks=-1.0) == 1


def rope(lib, bwd, q=A, qs=None, k=A, ks=None, cs=A, dim=64, max_pos=9, inter=0, pos=A, axes=2, pb=2, pair=AXES, qo=2 * A,
         qos=None, ko=2 * A, kos=None, B=2, H=4, Hkv=2, N=3, d=64):
    f = lib.attn_rope_axes_bwd if bwd else lib.attn_rope_axes
    return f(q, qs, k, ks, cs, dim, max_pos, inter, pos, axes, pb, pair, qo, qos, ko, kos, B, H, Hkv, N, d, None)


@pytest.mark.parametrize("bad, status", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(cs=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(Hkv=0), 1),
    (dict(B=0), 1), (dict(max_pos=0), 1), (dict(inter=3), 1), (dict(pb=3), 1), (dict(pos=None), 1),
    (dict(B=1 << 20, N=1 << 12, pb=1), 1), (dict(qo=A, qos=strides(768, 192, 64), qs=strides(768, 64, 256)), 1),
    (dict(qs=strides(-768, 64, 256)), 1), (dict(dim=80), 2), (dict(dim=0), 2), (dict(d=48, dim=48), 2), (dict(axes=5), 2),
    (dict(q=A + 8), 3), (dict(ko=A + 8), 3), (dict(cs=A + 4), 3), (dict(kos=strides(768, 64, 252)), 3),
])
@pytest.mark.parametrize("bwd", [False, True])
def test_rope_refusals(lib, bad, status, bwd):
    assert rope(lib, bwd, **bad) == status


def test_unpack_and_decode_refusals(lib):
    def unpack(k=A, v=A, ks=S, vs=S, ids=A, n=3, ko=A, vo=A, ps=16, Hkv=2, d=64, P=9):
        return lib.paged_kv_unpack_fp4(k, v, ks, vs, ids, n, ko, vo, ps, Hkv, d, P, None)
    for bad in (dict(k=None), dict(vo=None), dict(ids=None), dict(n=0), dict(P=0), dict(ks=0.0), dict(vs=-1.0)):
        assert unpack(**bad) == 1, bad
    assert unpack(d=72) == 2 and unpack(ps=8) == 2 and unpack(k=A + 4) == 3 and unpack(vo=A + 8) == 3 and unpack(ids=A + 2) == 3

    def decode(q=A, ks=S, vs=S, ps=16, B=2, H=4, Hkv=2, d=64, scale=0.1, cap=0.0, slopes=None, ws=A, n=1 << 30, kp=A):
        return lib.paged_attn_decode_fp4(q, kp, A, ks, vs, A, A, ps, A, None, B, H, Hkv, d, 8, 9, scale, cap, slopes, None, ws,
                                         n, None)
    for bad in (dict(q=None), dict(ks=0.0), dict(vs=float("nan")), dict(B=0), dict(Hkv=3), dict(scale=-1.0), dict(cap=-1.0),
                dict(cap=1e31), dict(scale=1e-30, slopes=A), dict(ks=1e-38)):
        assert decode(**bad) == 1, bad
    assert decode(d=48) == 2 and decode(ps=32) == 2 and decode(kp=A + 8) == 3 and decode(slopes=A + 2) == 3
    need = lib.paged_attn_decode_fp4_workspace_size(2, 4, 2, 64, 8, 16)
    assert need > 0 and decode(n=need - 1) == 4 and decode(ws=None) == 4 and decode(ws=A + 8) == 4
    assert lib.paged_attn_decode_fp4_workspace_size(2, 4, 2, 48, 8, 16) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    from attn_fwd_02_gb300 import binding as b
    z, i = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    pages, cs = torch.zeros(4, 2, 9 * 64, dtype=torch.uint8), torch.zeros(8, 64)
    pos = torch.zeros(2, 1, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        b.paged_kv_append_fp4(z, z, z, pages, pages, S, S, i[None], i, cos_sin=cs)
    with pytest.raises(ValueError):
        b.paged_kv_append_rope_axes(z, z, z, pages, pages, cs, pos, AXES, i[None], i)
    with pytest.raises(ValueError):
        b.attn_rope_axes(z, z, cs, pos, AXES)
    with pytest.raises(ValueError):
        b.paged_attn_decode_fp4(z[:, :, 0], pages, pages, S, S, i[None], i)
    with pytest.raises(ValueError):
        b.paged_kv_unpack_fp4(pages, pages, S, S, i)
    with pytest.raises(TypeError):
        b.paged_kv_unpack_fp4(pages.float(), pages, S, S, i)


@pytest.mark.parametrize("scale, k_scale", [(1e-10, 1e-30), (1e-30, 1e-20), (1e20, 1e30), (1e30, 1e9)])
def test_decode_refuses_scales_whose_product_leaves_fp32(lib, scale, k_scale):
    # a product of 0 or infinity would meet unseen scores of -infinity as NaN
    for slopes in (None, A):
        assert lib.paged_attn_decode_fp4(A, A, A, k_scale, S, A, A, 16, A, None, 2, 4, 2, 64, 8, 9, scale, 0.0, slopes, None, A,
                                         1 << 30, None) == 1
