"""Forking, reserving and compacting at the sizes where the work is cut another way (1024 and 8192 entries or pages), the table
and the pool each small and large, against their definition (pages_ref)."""
import random

import pytest
import torch

import pages_ref as R
from test_gpu_pages import dev, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attn_fwd_02_gb300 import binding, build
    build.build()
    return binding


SIZES = [(16, 64, 1024), (25, 41, 1023), (8, 9, 1025), (40, 60, 2048), (64, 128, 8192), (3, 2731, 300), (64, 64, 8193), (100, 80, 4096),
         (130, 250, 900), (2, 5, 32769)]  # B, W, P


@pytest.mark.parametrize("B, W, P", SIZES)
def test_fork_reserve_compact(lib, B, W, P):
    for seed, fill in ((1, 0.5), (2, 0.95)):
        r = random.Random(seed)
        table, ctx, ref = R.state(B, W, P, seed, fill)
        parents = [r.choice((b, r.randrange(B), -1)) for b in range(B)]
        new = [r.choice((0, 1, 1, r.randint(1, 60), 16 * W)) for _ in range(B)]
        forked = R.fork(table, ctx, parents, ref, P)
        got = R.reserve(*forked[:2], new, forked[2], P)
        moved = R.compact(*got[:2], P)
        t, c, n, p, a = dev(table, ctx, ref, parents, new)
        for in_place in (False, True):
            f = lib.paged_kv_fork(t, c, p, n, ref_counts_out=n if in_place else None)
            same(f, forked)
            f = [x.clone() for x in f]
            g = lib.paged_kv_reserve(f[0], f[1], a, f[2], *(f[0], f[2]) if in_place else ())
            same(g, got)
            same(lib.paged_kv_compact(g[0], g[1], g[0] if in_place else None), moved)
