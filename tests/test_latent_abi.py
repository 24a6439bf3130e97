"""Host checks of the latent cache and attention calls: every refusal comes
before any launch (fake non-null pointers, never dereferenced)."""
import ctypes
import os
import re
import subprocess

import pytest

import edge_moe_serving_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 256     # an aligned address


def cache(**k):
    v = dict(pages=A, table=A, lens=A, refs=A, n_layers=2, n_pages=100, page_tokens=64, rank=512, rope=64, max_seqs=8,
             max_blocks=16, reserved=0)
    v.update(k)
    return moe.moe_kv_cache(*v.values())


BAD_STRUCTS = [
    (dict(pages=None), moe.MOE_ERR_INVALID_ARG), (dict(table=None), moe.MOE_ERR_INVALID_ARG),
    (dict(lens=None), moe.MOE_ERR_INVALID_ARG), (dict(refs=None), moe.MOE_ERR_INVALID_ARG),
    (dict(n_layers=0), moe.MOE_ERR_INVALID_ARG), (dict(n_pages=0), moe.MOE_ERR_INVALID_ARG),
    (dict(rank=0), moe.MOE_ERR_INVALID_ARG), (dict(rope=-8), moe.MOE_ERR_INVALID_ARG),
    (dict(max_seqs=0), moe.MOE_ERR_INVALID_ARG), (dict(max_blocks=0), moe.MOE_ERR_INVALID_ARG),
    (dict(page_tokens=0), moe.MOE_ERR_INVALID_ARG),
    (dict(page_tokens=48), moe.MOE_ERR_UNSUPPORTED), (dict(page_tokens=256), moe.MOE_ERR_UNSUPPORTED),
    (dict(rank=516), moe.MOE_ERR_UNSUPPORTED), (dict(rope=4), moe.MOE_ERR_UNSUPPORTED),
    (dict(max_seqs=8193), moe.MOE_ERR_UNSUPPORTED), (dict(n_pages=1 << 25), moe.MOE_ERR_UNSUPPORTED),
    (dict(max_blocks=1 << 29), moe.MOE_ERR_UNSUPPORTED), (dict(pages=A + 8), moe.MOE_ERR_UNSUPPORTED),
    (dict(table=A + 2), moe.MOE_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", BAD_STRUCTS)
def test_every_call_checks_the_struct(change, status):
    L, c = moe.lib(), cache(**change)
    r = ctypes.byref(c)
    assert L.moe_kv_workspace_size(r, 4) == 0
    assert L.moe_kv_reserve(r, A, A, 1, A, 1 << 30, None, None) == status
    assert L.moe_kv_append(r, 0, A, A, A, 1, None, None) == status
    assert L.moe_kv_fork(r, A, A, 1, A, 1 << 30, None, None) == status
    assert L.moe_kv_free(r, A, 1, None, None) == status
    assert L.moe_kv_compact(r, None, A, 1 << 30, None, None) == status
    assert L.moe_latent_decode_workspace_size(r, 1, 1, 16, 0) == 0
    assert L.moe_latent_decode(r, 0, A, A, 1, 1, 16, 1.0, 0, A, None, A, 1 << 40, None, None) == status
    assert L.moe_latent_prefill_workspace_size(r, 1, 1, 16, 128, 128, 10) == 0
    assert L.moe_latent_prefill(r, 0, A, A, A, 1, 1, 16, 128, 128, A, 1.0, 10, A, A, 1 << 40, None, None) == status


def test_null_struct():
    L = moe.lib()
    assert L.moe_kv_free(None, A, 1, None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_workspace_size(None, 1) == 0


def test_page_calls_refuse():
    L, c = moe.lib(), cache()
    r = ctypes.byref(c)
    need = moe.moe_kv_workspace_size(c, 8)
    assert need >= 8 * 16 * 4 and moe.moe_kv_workspace_size(c, -1) == 0
    for call in (lambda n, a, ws, nb: L.moe_kv_reserve(r, a, A, n, ws, nb, None, None),
                 lambda n, a, ws, nb: L.moe_kv_fork(r, a, A, n, ws, nb, None, None)):
        assert call(-1, A, A, need) == moe.MOE_ERR_INVALID_ARG
        assert call(9, A, A, 1 << 30) == moe.MOE_ERR_INVALID_ARG      # more entries than sequences
        assert call(2, None, A, need) == moe.MOE_ERR_INVALID_ARG
        assert call(0, None, None, 0) == moe.MOE_OK
        assert call(8, A, A, 16) == moe.MOE_ERR_WORKSPACE
        assert call(8, A, None, need) == moe.MOE_ERR_WORKSPACE
        assert call(8, A, A + 64, need) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_kv_free(r, None, 1, None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_free(r, A, 9, None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_compact(r, None, A, 0, None, None) == moe.MOE_ERR_WORKSPACE
    assert L.moe_kv_append(r, 2, A, A, A, 1, None, None) == moe.MOE_ERR_INVALID_ARG     # layer
    assert L.moe_kv_append(r, 0, A, A, A, -1, None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_append(r, 0, None, A, A, 1, None, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_append(r, 0, A + 8, A, A, 1, None, None) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_kv_append(r, 0, None, None, None, 0, None, None) == moe.MOE_OK


def test_decode_refuses():
    L, c = moe.lib(), cache()
    r = ctypes.byref(c)

    def call(layer=0, q=A, seqs=A, B=4, Q=1, heads=16, scale=0.1, shared=0, out=A, ws=A, nb=1 << 40, c=r):
        return L.moe_latent_decode(c, layer, q, seqs, B, Q, heads, scale, shared, out, None, ws, nb, None, None)

    for bad in (dict(layer=2), dict(layer=-1), dict(B=-1), dict(Q=0), dict(heads=0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(shared=-64), dict(shared=32), dict(shared=17 * 64), dict(q=None),
                dict(seqs=None), dict(out=None)):
        assert call(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(B=4097), dict(Q=9, heads=128), dict(q=A + 8), dict(out=A + 8)):
        assert call(**bad) == moe.MOE_ERR_UNSUPPORTED, bad
    for change in (dict(rank=64), dict(rank=640), dict(rope=8), dict(rope=80)):
        assert call(c=ctypes.byref(cache(**change))) == moe.MOE_ERR_UNSUPPORTED
    assert call(B=0, q=None, seqs=None, out=None, ws=None, nb=0) == moe.MOE_OK
    need = moe.moe_latent_decode_workspace_size(c, 4, 1, 16, 64)
    assert need > 0 and moe.moe_latent_decode_workspace_size(c, 4, 9, 128, 0) == 0
    assert call(shared=64, nb=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(shared=64, ws=None, nb=need) == moe.MOE_ERR_WORKSPACE
    assert call(shared=64, ws=A + 16, nb=need) == moe.MOE_ERR_UNSUPPORTED
    assert call(c=ctypes.byref(cache(max_blocks=1 << 22, max_seqs=1))) == moe.MOE_ERR_UNSUPPORTED


def test_prefill_refuses():
    L, c = moe.lib(), cache()
    r = ctypes.byref(c)

    def call(layer=0, q=A, seqs=A, off=A, B=2, T=9, heads=16, dn=128, dv=128, w=A, scale=0.1, kv=100, out=A, ws=A,
             nb=1 << 40, c=r):
        return L.moe_latent_prefill(c, layer, q, seqs, off, B, T, heads, dn, dv, w, scale, kv, out, ws, nb, None, None)

    for bad in (dict(layer=2), dict(B=-1), dict(T=-1), dict(heads=0), dict(kv=-1), dict(scale=float("inf")),
                dict(q=None), dict(seqs=None), dict(off=None), dict(w=None), dict(out=None)):
        assert call(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(dn=96), dict(dv=192), dict(heads=1025), dict(B=4097), dict(T=1 << 28), dict(kv=1 << 28),
                dict(q=A + 8), dict(w=A + 8), dict(out=A + 2)):
        assert call(**bad) == moe.MOE_ERR_UNSUPPORTED, bad
    assert call(c=ctypes.byref(cache(rank=64))) == moe.MOE_ERR_UNSUPPORTED
    need = moe.moe_latent_prefill_workspace_size(c, 2, 9, 16, 128, 128, 100)
    assert need >= 16 * 100 * 256 * 2
    assert call(nb=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(ws=A + 16, nb=need) == moe.MOE_ERR_UNSUPPORTED
    assert call(B=0, T=0, q=None, seqs=None, off=None, w=None, out=None, ws=None, nb=0) == moe.MOE_OK
    assert call(T=0, q=None, out=None, ws=None, nb=0) == moe.MOE_OK


def test_struct_layout_equals_the_headers(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "moe.h"\nint main(void) { printf("%d %d %d\\n", (int)sizeof(moe_kv_cache),'
                   ' (int)offsetof(moe_kv_cache, n_layers), (int)offsetof(moe_kv_cache, max_blocks)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(moe.moe_kv_cache), moe.moe_kv_cache.n_layers.offset, moe.moe_kv_cache.max_blocks.offset]


def test_device_error_bits_are_the_headers():
    with open(os.path.join(ROOT, "include", "moe.h")) as f:
        src = f.read()
    for name in ("BAD_SEQ", "BAD_PAGE", "CAPACITY"):
        value = int(re.search(r"#define MOE_DEV_ERR_%s (\d+)u" % name, src).group(1))
        assert getattr(moe, "MOE_DEV_ERR_" + name) == value
