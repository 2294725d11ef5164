"""The rotation by several axes refuses outputs whose rows overlap one another: each row is a block's own (on the host: a status
before any device work)."""
import ctypes

import pytest

A = 1 << 20  # fake, 16-byte aligned addresses: the checks fail before any use
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    from attn_fwd_02_gb300 import binding
    from attn_fwd_02_gb300 import build as buildmod
    buildmod.build()
    return binding.load_library()


def strides(s):
    return None if s is None else (ctypes.c_int64 * 3)(*s)


def rope(lib, bwd, q=A, qs=None, ks=None, qo=2 * A, qos=None, k=A + 4096, ko=3 * A, kos=None, B=2, H=4, Hkv=2, N=3, d=64):
    f = lib.attn_rope_axes_bwd if bwd else lib.attn_rope_axes
    return f(q, strides(qs), k, strides(ks), A, d, 9, 0, A, 2, B, bytes([0, 1] * (d // 4)), qo, strides(qos), ko, strides(kos), B, H,
             Hkv, N, d, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("bad", [
    dict(qos=(0, 192, 64)), dict(qos=(768, 0, 64)), dict(qos=(768, 192, 0)), dict(qos=(0, 0, 0)),  # expanded
    dict(kos=(0, 192, 64)), dict(kos=(384, 0, 64)), dict(kos=(384, 192, 0)),
    dict(qos=(768, 192, 56)), dict(qos=(768, 184, 64)), dict(qos=(760, 192, 64)), dict(qos=(64, 192, 64)),  # into the next one
    dict(qos=(248, 64, 256)), dict(kos=(64, 128, 128)),
    dict(qos=(768, 8, 64)), dict(N=1, qos=(256, 56, 0)), dict(B=1, H=1 << 20, N=2, qos=(0, 64, 1 << 25)),
    dict(qs=(768, 0, 64), qo=A, qos=(768, 0, 64)),  # an expanded input in place
    dict(ko=2 * A),                                 # one place for both outputs
], ids=str)
def test_overlapping_rows(lib, bad, bwd):
    assert rope(lib, bwd, **bad) == INVALID
