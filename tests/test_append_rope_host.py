"""Host-side refusals of the append with rotation: bad arguments come back as a status before any
device work, and the binding's checks raise before the library is called."""
import ctypes

import pytest

A = 1 << 20  # fake, 16-byte aligned addresses: the checks fail before any use


@pytest.fixture(scope="module")
def lib():
    from attn_fwd_02_gb300 import binding
    from attn_fwd_02_gb300 import build as buildmod
    buildmod.build()
    return binding.load_library()


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def call(lib, q=A, qs=None, k=A, ks=None, v=A, vs=None, qo=A, kp=A, vp=A, cs=A, rope=64, max_pos=100, inter=0, table=A,
         start=A, new=None, ps=16, B=2, H=4, Hkv=2, N=3, d=64, max_pages=8, num_pages=9):
    return lib.paged_kv_append_rope(q, qs, k, ks, v, vs, qo, kp, vp, cs, rope, max_pos, inter, table, start, new, ps, B,
                                    H, Hkv, N, d, max_pages, num_pages, None)


@pytest.mark.parametrize("bad, status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(cs=None), 1),
    (dict(table=None), 1), (dict(start=None), 1), (dict(q=None), 1), (dict(qo=None), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(Hkv=-1), 1), (dict(N=0), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1),
    (dict(max_pos=0), 1), (dict(inter=2), 1), (dict(B=1 << 20, N=1 << 12), 1), (dict(max_pages=1 << 27), 1),
    (dict(qs=strides(-768, 64, 256)), 1),
    (dict(d=48, rope=48), 2), (dict(ps=32), 2), (dict(rope=0), 2), (dict(rope=72), 2), (dict(rope=80), 2),
    (dict(q=A + 2), 3), (dict(qo=A + 8), 3), (dict(k=A + 4), 3), (dict(cs=A + 4), 3), (dict(vp=A + 8), 3),
    (dict(table=A + 2), 3), (dict(new=A + 1), 3), (dict(ks=strides(768, 68, 256)), 3), (dict(vs=strides(766, 64, 256)), 3),
])
def test_refusals(lib, bad, status):
    assert call(lib, **bad) == status


def test_fp8_scales_are_checked(lib):
    for ks, vs in ((0.0, 1.0), (1.0, float("nan")), (-1.0, 1.0), (float("inf"), 1.0)):
        assert lib.paged_kv_append_rope_fp8(A, None, A, None, A, None, A, A, A, ks, vs, A, 64, 100, 0, A, A, None, 16, 2,
                                            4, 2, 3, 64, 8, 9, None) == 1


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    from attn_fwd_02_gb300 import binding
    z = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.paged_kv_append_rope(z, z, z, pages, pages, torch.zeros(8, 64), i[None], i)
    with pytest.raises(TypeError):
        binding.paged_kv_append_rope(z, z.float(), z, pages, pages, torch.zeros(8, 64), i[None], i)
