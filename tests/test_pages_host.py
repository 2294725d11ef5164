"""Refusals of the calls on page tables, counts and pages, and the reference's own invariants, on the host."""
import ctypes

import pytest
import torch

import pages_ref as R

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from attn_fwd_02_gb300 import binding
    from attn_fwd_02_gb300 import build as buildmod
    buildmod.build()
    return binding.load_library()


def test_reference_keeps_one_count_per_entry():
    for seed in range(20):
        P, B, W = 60, 7, 9
        table, ctx, ref = R.state(B, W, P, seed)
        table, ctx, ref = R.fork(table, ctx, [1, 1, -1, 3, 0, 5, 99, 2], ref, P)
        table, ref, got, src, dst = R.reserve(table, ctx, [1, 0, 30, 1, 17, 1, 1, 400], ref, P)
        table, ref, s, d, n = R.compact(table, ref, P)
        count = [0] * P
        for row in table:
            for e in row:
                if e >= 0:
                    count[e] += 1
        assert count == ref and sum(1 for c in ref if c) == (max((i for i in range(P) if ref[i]), default=-1) + 1)


def test_fork_refusals(lib):
    def f(t=A, c=A, p=A, r=A, to=2 * A, co=2 * A, ro=2 * A, ps=16, B=2, Bo=3, W=4, P=9):
        return lib.paged_kv_fork(t, c, p, r, to, co, ro, ps, B, Bo, W, P, None)
    for bad in (dict(t=None), dict(p=None), dict(ro=None), dict(B=0), dict(Bo=0), dict(W=0), dict(P=-1), dict(to=A), dict(co=A),
                dict(W=1 << 27), dict(p=3 * A, co=3 * A)):
        assert f(**bad) == 1, bad
    assert f(ps=32) == 2 and f(t=A + 2) == 3 and f(ro=A + 1) == 3


def test_reserve_refusals(lib):
    def f(t=A, c=A, n=A, r=A, to=A, ro=A, got=A, s=A, d=A, ps=16, B=2, W=4, P=9, ws=A, size=1 << 20):
        return lib.paged_kv_reserve(t, c, n, r, to, ro, got, s, d, ps, B, W, P, ws, size, None)
    for bad in (dict(c=None), dict(n=None), dict(got=None), dict(d=None), dict(B=0), dict(P=0), dict(W=1 << 27)):
        assert f(**bad) == 1, bad
    need = lib.paged_kv_reserve_workspace_size(2, 9)
    assert f(ps=8) == 2 and f(r=A + 4) == 3 and f(ro=A + 8) == 3 and f(s=A + 2) == 3
    assert need > 0 and f(size=need - 1) == 4 and f(ws=None) == 4 and f(ws=A + 4) == 4
    assert lib.paged_kv_reserve_workspace_size(0, 9) == 0 and lib.paged_kv_compact_workspace_size(0) == 0


def test_compact_and_copy_refusals(lib):
    def f(t=A, r=A, to=A, ro=2 * A, s=A, d=A, n=A, B=2, W=4, P=9, ws=A, size=1 << 20):
        return lib.paged_kv_compact(t, r, to, ro, s, d, n, B, W, P, ws, size, None)
    for bad in (dict(t=None), dict(n=None), dict(B=0), dict(P=0), dict(ro=A)):
        assert f(**bad) == 1, bad
    assert f(r=A + 4) == 3 and f(d=A + 2) == 3 and f(size=lib.paged_kv_compact_workspace_size(9) - 1) == 4

    def c(pools=(A, A), size=512, s=A, d=A, count=None, n=3, P=9, n_pools=None):
        at = (ctypes.c_void_p * max(1, len(pools)))(*pools)
        return lib.paged_kv_copy_pages(at, len(pools) if n_pools is None else n_pools, size, s, d, count, n, P, None)
    for bad in (dict(pools=(A, None)), dict(n_pools=0), dict(size=0), dict(size=24), dict(s=None), dict(n=0), dict(P=0)):
        assert c(**bad) == 1, bad
    assert c(pools=(A, A + 8)) == 3 and c(count=A + 2) == 3 and c(s=A + 1) == 3


def test_binding_refuses_cpu_tensors_and_wrong_pools():
    from attn_fwd_02_gb300 import binding as b
    t, i = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: b.paged_kv_fork(t, i, i, i), lambda: b.paged_kv_reserve(t, i, i, i), lambda: b.paged_kv_compact(t, i),
                 lambda: b.paged_kv_copy_pages([t], i, i)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        b.paged_kv_fork(t.float(), i, i, i)


@pytest.mark.parametrize("B, W, P", [(1 << 20, 1 << 11, 9), (64, 1 << 26, 9), (2, 4, (1 << 30) + 1), (2, 4, 2**31 - 1)])
def test_tables_and_pools_past_32_bit_sums_are_refused(lib, B, W, P):
    z = 1 << 62  # (a workspace's size is not what fails)
    assert lib.paged_kv_fork(A, A, A, A, 2 * A, 2 * A, 2 * A, 16, B, 1, W, P, None) == 1
    assert lib.paged_kv_reserve(A, A, A, A, A, A, A, A, A, 16, B, W, P, A, z, None) == 1
    assert lib.paged_kv_compact(A, A, A, 2 * A, A, A, A, B, W, P, A, z, None) == 1
    if P == 9:
        assert lib.paged_kv_fork(A, A, A, A, 2 * A, 2 * A, 2 * A, 16, 1, B, W, P, None) == 1
