"""Attention weights of rows that looked at nothing: their log-sum-exp is -infinity
and they add nothing, whatever their scores are."""
import math

import pytest
import torch

import edge_moe_serving_gb300 as moe
from fp4_helpers import Paged4
from kv_helpers import DEV, Paged
from test_gpu_latent_attention import make_q, run_decode
from test_gpu_latent_weights import check, lse64, run_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,Q", [(16, 1), (20, 4), (65, 2), (128, 3)])
@pytest.mark.parametrize("four", [False, True])
def test_rows_without_a_sum_add_nothing(heads, Q, four):
    lens = [300, 1, 129, 40]
    c = (Paged4 if four else Paged)(20, 32, 256, 32, 4, 11)
    rows = c.fill(lens, seed=heads)
    q = make_q(4 * Q, heads, c.row, 7)
    lse = lse64(rows, q, [0, 1, 2, 3], Q, heads, 0.1)
    g = torch.Generator().manual_seed(heads)
    gone = (torch.rand(lse.shape, generator=g) < 0.3).to(DEV)
    gone[2 * Q:3 * Q] = True                                # every row of a sequence
    old = torch.rand(4, 11 * 32, device=DEV)
    lse[gone] = -math.inf
    got = run_weights(c, q, [0, 1, 2, 3], Q, heads, 0.1, lse, 0.5, old.clone())
    assert c.bits() == 0
    lse[gone] = math.inf                                    # to the definition in 64 bits: exp(s - infinity) = 0
    check(rows, q, [0, 1, 2, 3], Q, heads, 0.1, lse, 0.5, old, got)


def test_after_a_decode_whose_prefix_has_no_sequence():
    """A bad first id with shared tokens gives every row zeros and lse = -inf; the weights of the others only fade."""
    c = Paged(20, 64, 512, 64, 3, 6)
    c.fill([200, 130, 300], seed=9)
    q = make_q(3, 16, c.row, 8)
    _, lse = run_decode(c, q, [-1, 0, 2], 1, 16, 0.07, shared=64)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ and bool((lse == -math.inf).all())
    old = torch.rand(3, 6 * 64, device=DEV)
    got = run_weights(c, q, [-1, 0, 2], 1, 16, 0.07, lse, 0.5, old.clone())
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    want = old.clone()
    for s, n in ((0, 200), (2, 300)):
        want[s, :n] *= 0.5
    assert torch.equal(got, want)


def test_every_token_left_out():
    """Infinite rotary entries that make all of a sequence's scores -infinity: the answer is zeros, the weights are too."""
    c = Paged(12, 32, 128, 16, 2, 4)
    c.fill([70, 60], seed=11)
    q = make_q(2, 4, c.row, 12)
    q[0, :, 128:] = -1.0
    q[0, :, 129:] = 0.0
    for b in range(3):
        c.pages[0, int(c.table[0, b]), :, 128] = math.inf   # q . row = -infinity for sequence 0
    out, lse = run_decode(c, q, [0, 1], 1, 4, 0.1)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    got = run_weights(c, q, [0, 1], 1, 4, 0.1, lse, 1.0, torch.zeros(2, 128, device=DEV))
    assert c.bits() == 0 and bool((got[0] == 0).all())
    assert abs(float(got[1].double().sum()) - 4) <= 4 * 2.0 ** -10
