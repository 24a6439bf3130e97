"""Workspaces of the latent attention calls: one made for the largest call
serves every smaller one (sizes alone, no GPU)."""
import random

import pytest

import edge_moe_serving_gb300 as moe


def cache(**k):
    v = dict(pages=256, table=256, lens=256, refs=256, n_layers=1, n_pages=4096, page_tokens=64, rank=512, rope=64,
             max_seqs=600, max_blocks=1024, reserved=0)
    v.update(k)
    return moe.moe_kv_cache(*v.values())


@pytest.mark.parametrize("heads,dn,dv,kv", [(16, 128, 128, 16384), (1, 64, 128, 5000), (128, 128, 64, 70000), (8, 64, 64, 300)])
def test_prefill_size_never_falls_with_the_queries(heads, dn, dv, kv):
    c = cache()
    for B in (1, 2, 7, 40):
        sizes = [moe.moe_latent_prefill_workspace_size(c, B, T, heads, dn, dv, kv) for T in range(1, 20000, 37)]
        assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("shared", [0, 1024])
@pytest.mark.parametrize("heads", [1, 5, 16, 20, 72, 128])
def test_decode_size_never_falls_with_the_batch(heads, shared):
    c = cache()
    for Q in (1, 2, 5):
        sizes = [moe.moe_latent_decode_workspace_size(c, B, Q, heads, shared) for B in range(1, 560)]
        assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_any_smaller_call_fits():
    rng = random.Random(1)
    for _ in range(3000):
        c = cache(rank=rng.choice([128, 256, 384, 512]), rope=rng.choice([0, 16, 64]))
        heads, dn, dv = rng.choice([1, 2, 8, 16, 20, 37, 128]), rng.choice([64, 128]), rng.choice([64, 128])
        B, T, kv = rng.randint(1, 50), rng.randint(1, 9000), rng.randint(1, 60000)
        b, t, k = rng.randint(1, B), rng.randint(1, T), rng.randint(1, kv)
        size = moe.moe_latent_prefill_workspace_size
        assert 0 < size(c, b, t, heads, dn, dv, k) <= size(c, B, T, heads, dn, dv, kv), (heads, dn, dv, B, T, kv, b, t, k)
        Q = rng.randint(1, 1024 // heads)
        q, h, shared = rng.randint(1, Q), rng.randint(1, heads), 64 * rng.randint(0, 500)
        size = moe.moe_latent_decode_workspace_size
        assert 0 < size(c, b, q, h, rng.choice([0, shared])) <= size(c, B, Q, heads, shared), (B, Q, heads, shared, b, q, h)
        n = rng.randint(0, 600)
        assert moe.moe_kv_workspace_size(c, rng.randint(0, n)) <= moe.moe_kv_workspace_size(c, n)
