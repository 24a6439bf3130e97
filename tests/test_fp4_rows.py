"""The 4-bit row's packing in the tests' own look-up form, and the host checks of
the calls over 4-bit caches, attention weights and eviction (no GPU: every
refusal comes before any launch)."""
import ctypes

import numpy as np
import pytest
import torch

import edge_moe_serving_gb300 as moe
from fp4_helpers import SCALES, SIZES, pack, row_bytes, unpack
from test_latent_abi import A, BAD_STRUCTS, cache


def fp4(**k):
    return cache(**{**dict(reserved=moe.MOE_KV_FP4), **k})


def test_scales_are_f16_shifted():
    bits = (np.arange(248, dtype=np.int32) << 7).astype(np.int16)
    assert np.array_equal(SCALES, torch.from_numpy(bits).view(torch.float16).double().numpy())


def test_every_value_is_a_bf16():
    v = torch.from_numpy(np.outer(SCALES, SIZES))
    assert torch.equal(v.to(torch.bfloat16).double(), v)


def test_pack_is_idempotent_and_near():
    g = torch.Generator().manual_seed(1)
    rows = (torch.randn(300, 256 + 32, generator=g) * torch.exp(3 * torch.randn(300, 1, generator=g))).to(torch.bfloat16)
    data = pack(rows, 256, 32)
    values = unpack(data, 256, 32)
    assert torch.equal(values[:, 256:], rows[:, 256:].double())
    lat, got = rows[:, :256].double().view(300, 16, 16), values[:, :256].view(300, 16, 16)
    top = lat.abs().amax(-1, keepdim=True)
    # half a step of the largest code is 1/6 of the largest value, and the scale's own rounding 2^-4 of it
    assert bool(((lat - got).abs() <= top * (1 / 6 + 2.0 ** -4)).all())
    # stored again: the same scale where the largest code is 6, and then the same codes
    full = got.abs().amax(-1) == 6 * torch.from_numpy(SCALES[data[:, 256 // 2 + 64:256 // 2 + 64 + 16].numpy()])
    again = unpack(pack(values.to(torch.bfloat16), 256, 32), 256, 32)[:, :256].view(300, 16, 16)
    assert bool(full.any()) and torch.equal(again[full], got[full])


@pytest.mark.parametrize("rank,rope", [(512, 64), (512, 0), (256, 32), (128, 64), (384, 16), (32, 8), (96, 0)])
def test_row_bytes(rank, rope):
    assert moe.moe_kv_row_bytes(rank, rope, moe.MOE_KV_FP4) == row_bytes(rank, rope)
    assert moe.moe_kv_row_bytes(rank, rope, moe.MOE_KV_BF16) == 2 * (rank + rope)


def test_row_bytes_refuses():
    for rank, rope, fmt in ((0, 0, 0), (512, -8, 0), (12, 0, 0), (512, 4, 1), (48, 0, 1), (512, 64, 2), (512, 64, -1),
                            (1 << 20, 8, 0)):
        assert moe.moe_kv_row_bytes(rank, rope, fmt) == 0, (rank, rope, fmt)


STRUCTS = BAD_STRUCTS + [(dict(reserved=2), moe.MOE_ERR_INVALID_ARG), (dict(reserved=-1), moe.MOE_ERR_INVALID_ARG),
                         (dict(rank=528), moe.MOE_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("change,status", STRUCTS)
def test_every_call_checks_the_struct(change, status):
    L, c = moe.lib(), fp4(**change)
    r = ctypes.byref(c)
    assert L.moe_kv_workspace_size(r, 4) == 0
    assert L.moe_kv_reserve(r, A, A, 1, A, 1 << 30, None, None) == status
    assert L.moe_kv_append(r, 0, A, A, A, 1, None, None) == status
    assert L.moe_kv_read(r, 0, A, A, 1, A, None, None) == status
    assert L.moe_kv_fork(r, A, A, 1, A, 1 << 30, None, None) == status
    assert L.moe_kv_free(r, A, 1, None, None) == status
    assert L.moe_kv_compact(r, None, A, 1 << 30, None, None) == status
    assert L.moe_kv_evict_workspace_size(r, 1) == 0
    assert L.moe_kv_evict(r, A, 1, A, 8, 0, 0, None, A, 1 << 40, None, None) == status
    assert L.moe_latent_decode(r, 0, A, A, 1, 1, 16, 1.0, 0, A, None, A, 1 << 40, None, None) == status
    assert L.moe_latent_prefill(r, 0, A, A, A, 1, 1, 16, 128, 128, A, 1.0, 10, A, A, 1 << 40, None, None) == status
    assert L.moe_latent_weights_workspace_size(r, 1, 1, 16) == 0
    assert L.moe_latent_weights(r, 0, A, A, 1, 1, 16, 1.0, A, 1.0, A, A, 1 << 40, None, None) == status


def test_read_refuses():
    L, c = moe.lib(), fp4()
    r = ctypes.byref(c)
    assert L.moe_kv_read(r, 2, A, A, 1, A, None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_read(r, -1, A, A, 1, A, None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_read(r, 0, A, A, -1, A, None, None) == moe.MOE_ERR_INVALID_ARG
    for args in ((None, A, A), (A, None, A), (A, A, None)):
        assert L.moe_kv_read(r, 0, args[0], args[1], 1, args[2], None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_read(r, 0, A, A, 1, A + 8, None, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_kv_read(r, 0, None, None, 0, None, None, None) == moe.MOE_OK


def test_weights_refuse():
    L, c = moe.lib(), fp4()
    r = ctypes.byref(c)

    def call(layer=0, q=A, seqs=A, B=4, Q=1, heads=16, scale=0.1, lse=A, decay=1.0, w=A, ws=A, nb=1 << 40, c=r):
        return L.moe_latent_weights(c, layer, q, seqs, B, Q, heads, scale, lse, decay, w, ws, nb, None, None)

    for bad in (dict(layer=2), dict(layer=-1), dict(B=-1), dict(Q=0), dict(heads=0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=None), dict(seqs=None), dict(lse=None), dict(w=None), dict(decay=-0.1),
                dict(decay=1.5), dict(decay=float("nan"))):
        assert call(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(B=4097), dict(Q=9, heads=128), dict(q=A + 8), dict(lse=A + 2), dict(w=A + 1)):
        assert call(**bad) == moe.MOE_ERR_UNSUPPORTED, bad
    for change in (dict(rank=64), dict(rank=640), dict(rope=8), dict(rope=80)):
        assert call(c=ctypes.byref(fp4(**change))) == moe.MOE_ERR_UNSUPPORTED
    assert call(B=0, q=None, seqs=None, lse=None, w=None, ws=None, nb=0) == moe.MOE_OK
    need = moe.moe_latent_weights_workspace_size(c, 4, 2, 64)
    assert need > 0 and moe.moe_latent_weights_workspace_size(c, 4, 9, 128) == 0
    assert call(Q=2, heads=64, nb=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(ws=A + 16) == moe.MOE_ERR_UNSUPPORTED
    assert call(ws=None) == moe.MOE_ERR_WORKSPACE


def test_evict_refuses():
    L, c = moe.lib(), fp4()
    r = ctypes.byref(c)
    need = moe.moe_kv_evict_workspace_size(c, 8)
    assert need > 0 and moe.moe_kv_evict_workspace_size(c, -1) == 0

    def call(seqs=A, n=4, w=A, budget=64, first=4, recent=16, kept=None, ws=A, nb=need, c=r):
        return L.moe_kv_evict(c, seqs, n, w, budget, first, recent, kept, ws, nb, None, None)

    for bad in (dict(n=-1), dict(n=9), dict(budget=0), dict(budget=-5), dict(first=-1), dict(recent=-1),
                dict(first=50), dict(recent=61), dict(first=1 << 30, recent=1 << 30, budget=(1 << 31) - 1),
                dict(seqs=None), dict(w=None)):
        assert call(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(w=A + 2), dict(kept=A + 1), dict(ws=A + 16),
                dict(c=ctypes.byref(fp4(max_seqs=4, max_blocks=(1 << 14) + 1)), nb=1 << 50)):
        assert call(**bad) == moe.MOE_ERR_UNSUPPORTED, bad
    assert call(nb=16) == moe.MOE_ERR_WORKSPACE and call(ws=None) == moe.MOE_ERR_WORKSPACE
    assert call(n=0, seqs=None, w=None, ws=None, nb=0) == moe.MOE_OK
    sizes = [moe.moe_kv_evict_workspace_size(c, n) for n in range(9)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("heads", [1, 16, 20, 64])
def test_decode_size_never_falls(heads):
    c = fp4(max_blocks=1024, max_seqs=600)
    for shared in (0, 1024, 16384, 65536):
        for Q in (1, 2, 5):
            sizes = [moe.moe_latent_decode_workspace_size(c, B, Q, heads, shared) for B in range(1, 560)]
            assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
    sizes = [moe.moe_latent_decode_workspace_size(c, 64, 1, heads, 64 * n) for n in range(1025)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_weights_size_never_falls():
    c = fp4()
    for a, b in (((1, 1, 8), (4, 1, 8)), ((4, 1, 8), (4, 8, 8)), ((4, 8, 8), (4, 8, 128)), ((4, 1, 64), (600, 1, 65))):
        assert 0 < moe.moe_latent_weights_workspace_size(c, *a) <= moe.moe_latent_weights_workspace_size(c, *b)
