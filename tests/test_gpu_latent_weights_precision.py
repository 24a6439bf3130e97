"""Attention weights keep fp32 all the way: their root-mean-square error, relative to
the definition in 64 bits.

A score is 576 products of bf16 values, exact, added in fp32 in steps of 16; let every
addend of a step (16 products and the running sum) be cut at 2^-24 of the largest magnitude M
in the step, all in one direction, which is the worst there is: 36 x 17 cuts of 2^-25 M on
average.  With entries of size one, |q . row| has a spread of sqrt(576) = 24, and M stays below 32
for all but one running sum in five, so 612 x 2^-25 x 32 x scale (0.07) = 2^-14.5 of a term.  lse
as given adds 2^-24 |lse| (|lse| < 16: 2^-20), the exponential 2^-22, a sum of fp32 terms in pairs less than 2^-20.
2^-14 covers them.  Operands or scores held in 11 bits (f16, tf32) would be off by 2^-12 / sqrt(3)
of scores of 2 to 4, which is 2^-11.5: eight times too much."""
import pytest
import torch

from fp4_helpers import Paged4
from kv_helpers import DEV, Paged
from test_gpu_latent_attention import make_q
from test_gpu_latent_weights import lse64, run_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("heads,Q", [(16, 1), (64, 1), (128, 1), (32, 16)])
def test_error(heads, Q, four):
    c = (Paged4 if four else Paged)(60, 64, 512, 64, 2, 40)
    rows = c.fill([2300, 700], seed=heads)
    q, scale = make_q(2 * Q, heads, c.row, 3), 0.07
    lse = lse64(rows, q, [0, 1], Q, heads, scale)
    assert float(lse.abs().max()) < 16
    got = run_weights(c, q, [0, 1], Q, heads, scale, lse, 0.0, torch.zeros(2, 40 * 64, device=DEV))
    assert c.bits() == 0
    for s, x in enumerate(rows):
        z = q[s * Q:(s + 1) * Q].cpu().double().reshape(Q * heads, -1) @ x.T * scale - lse[s * Q:(s + 1) * Q].cpu().double().view(-1, 1)
        limit = torch.tensor([len(x) - Q + i + 1 for i in range(Q) for _ in range(heads)])
        want = torch.exp(z).masked_fill(torch.arange(len(x)) >= limit[:, None], 0.0).sum(0)
        off = (got[s, :len(x)].cpu().double() - want) / want
        assert float(off.square().mean().sqrt()) <= 2.0 ** -14, float(off.square().mean().sqrt())
