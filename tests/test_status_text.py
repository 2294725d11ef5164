"""The text of a status names every reason that gives it."""
import pytest

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from attn_fwd_02_gb300 import binding
    from attn_fwd_02_gb300 import build as buildmod
    buildmod.build()
    return binding.load_library()


def text(lib, status):
    s = lib.attn_status_string(status)
    return s.decode() if isinstance(s, bytes) else s


def test_unsupported_names_the_rotation_and_no_limit_that_is_not_there(lib):
    # a rotation of 24 of 96 dims is refused as unsupported ...
    assert lib.paged_kv_append_rope(A, None, A, None, A, None, A, A, A, A, 24, 100, 0, A, A, None, 16, 2, 4, 2, 3, 96, 8, 9, None) == 2
    # ... and a backward at head dim 32, 80 or 96 is not (its workspace is what is wrong here)
    for d in (32, 80, 96):
        assert lib.attn_bwd(A, A, A, A, A, A, A, A, A, 1, 2, 2, 8, 8, d, 0, 0.1, None, None, 0, None) == 4
    s = text(lib, 2)
    assert "multiple of 16" in s and "backward" not in s
    for d in (32, 64, 80, 96, 128):
        assert str(d) in s
