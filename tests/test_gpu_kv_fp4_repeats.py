"""Attention and weights over 4-bit pages give the same bits on every run: many
tiles a CTA, so that every buffer is expanded into, multiplied and taken again
while the next tiles' codes arrive."""
import pytest
import torch

import edge_moe_serving_gb300 as moe
from fp4_helpers import Paged4
from kv_helpers import DEV
from test_gpu_latent_attention import make_q, make_w, run_decode, run_prefill
from test_gpu_latent_weights import run_weights

pytestmark = pytest.mark.gpu

RUNS = 20


def held(lens, page, rank, rope):
    c = Paged4(sum(-(-n // page) for n in lens) + 3, page, rank, rope, len(lens), max(-(-n // page) for n in lens) + 1)
    c.fill(lens, seed=rank)
    return c


@pytest.mark.parametrize("heads,Q", [(16, 1), (64, 1), (20, 2)])
def test_decode(heads, Q):
    c = held([40001, 333, 20000, 64], 64, 512, 64)
    q = make_q(4 * Q, heads, c.row, 3)
    first = run_decode(c, q, [0, 1, 2, 3], Q, heads, 0.07)
    assert all(bool(torch.isfinite(x).all()) for x in first)
    for _ in range(RUNS):
        for a, b in zip(first, run_decode(c, q, [0, 1, 2, 3], Q, heads, 0.07)):
            assert torch.equal(a, b)
    assert c.bits() == 0


@pytest.mark.parametrize("heads,Q", [(16, 1), (64, 1), (100, 1), (64, 8)])
def test_weights(heads, Q):
    c = held([40001, 333, 20000, 64], 64, 512, 64)
    q = make_q(4 * Q, heads, c.row, 4)
    _, lse = run_decode(c, q, [0, 1, 2, 3], Q, heads, 0.07)
    old = torch.zeros(4, c.table.shape[1] * 64, device=DEV)
    first = run_weights(c, q, [0, 1, 2, 3], Q, heads, 0.07, lse, 1.0, old.clone())
    assert bool(torch.isfinite(first).all())
    for _ in range(RUNS):
        assert torch.equal(first, run_weights(c, q, [0, 1, 2, 3], Q, heads, 0.07, lse, 1.0, old.clone()))
    assert c.bits() == 0


def test_prefill():
    c = held([5000, 700], 64, 512, 64)
    q, w = make_q(500, 8, 192, 5), make_w(8, 256, 512, 6)
    first = run_prefill(c, q, [0, 1], [0, 300, 500], 8, 128, 128, w, 0.07, 5700)
    for _ in range(RUNS):
        assert torch.equal(first, run_prefill(c, q, [0, 1], [0, 300, 500], 8, 128, 128, w, 0.07, 5700))
    assert c.bits() == 0
