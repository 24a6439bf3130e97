"""Attention weights of cached tokens against the definition in 64 bits.

A term is exp(s - lse): s carries at most 2^-24 sqrt(576) sum|q||k| scale < 2^-13 at
these spreads (products exact, sums fp32), lse as given 2^-24 of itself, the
exponential 2^-22 of itself; the sum of up to 1024 positive terms adds 2^-14 of
itself at most.  2^-11 covers them together; decay * old is rounded twice, 2^-23."""
import math

import pytest
import torch

import edge_moe_serving_gb300 as moe
from fp4_helpers import Paged4
from kv_helpers import DEV, Paged, attend64
from test_gpu_latent_attention import make_q, run_decode

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def run_weights(c, q, seqs, Q, heads, scale, lse, decay, weights, layer=0, stream=None):
    n = moe.moe_latent_weights_workspace_size(c.handle, len(seqs), Q, heads)
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device=DEV)
    moe.moe_latent_weights(c.handle, layer, q, i32(seqs), len(seqs), Q, heads, scale, lse, decay, weights, ws, ws.numel(),
                           c.status, stream)
    return weights


def lse64(rows, q, seqs, Q, heads, scale):
    out = []
    for b, s in enumerate(seqs):
        qb = q[b * Q:(b + 1) * Q].cpu().double().reshape(Q * heads, -1)
        limit = [len(rows[s]) - Q + i + 1 for i in range(Q) for _ in range(heads)]
        out.append(attend64(qb, rows[s], rows[s][:, :1], scale, limit)[2])
    return torch.stack(out).float().view(len(seqs) * Q, heads).to(DEV)


def check(rows, q, seqs, Q, heads, scale, lse, decay, old, got):
    seen = set()
    for b, s in enumerate(seqs):
        x = rows[s]
        seen.add(s)
        qb = q[b * Q:(b + 1) * Q].cpu().double().reshape(Q * heads, -1)
        z = (qb @ x.T) * scale - lse[b * Q:(b + 1) * Q].cpu().double().reshape(-1, 1)
        limit = torch.tensor([len(x) - Q + i + 1 for i in range(Q) for _ in range(heads)])
        p = torch.exp(z).masked_fill(torch.arange(len(x))[None] >= limit[:, None], 0.0).sum(0)
        before = old[s, :len(x)].cpu().double()
        ref = p + (decay * before if decay else 0.0)
        g = got[s, :len(x)].cpu().double()
        bound = 2.0 ** -11 * p + 2.0 ** -23 * (ref.abs() if decay else 0.0) + 1e-30
        assert bool(((g - ref).abs() <= bound).all()), (b, s, float(((g - ref).abs() / bound).max()))
        assert torch.equal(got[s, len(x):], old[s, len(x):])
    for s in range(old.shape[0]):
        if s not in seen:
            assert torch.equal(got[s], old[s])


CASES = [
    # rank, rope, page, heads, Q, lens, decay
    (512, 64, 64, 16, 1, [1], 1.0),
    (512, 64, 16, 64, 1, [1, 2, 127, 128, 129, 700, 333, 0], 0.5),
    (512, 64, 128, 20, 1, [300, 1, 129, 128, 1000], 1.0),
    (512, 64, 32, 8, 2, [2, 33, 95, 1], 0.0),              # a query that sees nothing
    (256, 32, 64, 48, 3, [5, 200, 64, 3], 0.9),
    (128, 0, 16, 1, 1, [1, 40, 16], 1.0),
    (384, 16, 32, 37, 4, [77, 4, 400], 1.0),
    (512, 64, 64, 128, 1, [640, 65], 0.25),
    (512, 64, 64, 32, 32, [2000], 1.0),                    # the last tokens of a prompt
    (512, 64, 64, 128, 8, [150, 8, 1029, 0], 1.0),
    (256, 48, 128, 7, 5, [0, 5, 0, 130], 1.0),
    (512, 0, 16, 65, 1, [70, 260], 1.0),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("rank,rope,page,heads,Q,lens,decay", CASES)
def test_weights(rank, rope, page, heads, Q, lens, decay, four):
    blocks = [-(-n // page) for n in lens]
    c = (Paged4 if four else Paged)(sum(blocks) + 5, page, rank, rope, len(lens) + 2, max(blocks) + 1)
    rows = c.fill(lens, seed=heads)
    q = make_q(len(lens) * Q, heads, c.row, 3)
    scale = 1.0 / math.sqrt(128 + rope)
    seqs = list(range(len(lens)))[::-1]
    lse = lse64(rows, q, seqs, Q, heads, scale)
    old = torch.rand(len(lens) + 2, c.table.shape[1] * page, device=DEV) * 3
    if decay == 0.0:
        old[:] = float("nan")                              # not read
        got = run_weights(c, q, seqs, Q, heads, scale, lse, decay, old.clone())
        old = torch.nan_to_num(old, nan=7.0)
        got = torch.where(torch.isnan(got), torch.full_like(got, 7.0), got)
    else:
        got = run_weights(c, q, seqs, Q, heads, scale, lse, decay, old.clone())
    assert c.bits() == 0
    check(rows, q, seqs, Q, heads, scale, lse, decay, old, got)
    if decay:
        assert torch.equal(got, run_weights(c, q, seqs, Q, heads, scale, lse, decay, old.clone()))   # the same bits


@pytest.mark.parametrize("heads,Q", [(16, 1), (65, 1), (128, 1), (100, 2)])
@pytest.mark.parametrize("four", [False, True])
def test_several_tiles_of_a_sequence_in_turn(heads, Q, four):
    """More than 152 x 128 tokens: every CTA takes tile after tile, with queries that stay, that do not in one pass, in several."""
    n = 45000
    c = (Paged4 if four else Paged)(-(-n // 128) + 1, 128, 128, 16, 2, -(-n // 128))
    rows = c.fill([n, 70], seed=heads)
    q = make_q(2 * Q, heads, c.row, 3)
    lse = lse64(rows, q, [1, 0], Q, heads, 0.1)
    old = torch.rand(2, c.table.shape[1] * 128, device=DEV)
    got = run_weights(c, q, [1, 0], Q, heads, 0.1, lse, 0.5, old.clone())
    assert c.bits() == 0
    check(rows, q, [1, 0], Q, heads, 0.1, lse, 0.5, old, got)


@pytest.mark.parametrize("four", [False, True])
def test_with_the_decode_calls_lse(four):
    """One step as it is used: the weights of a step sum to queries x heads."""
    c = (Paged4 if four else Paged)(60, 64, 512, 64, 3, 40)
    lens = [2303, 320, 77]
    c.fill(lens, seed=5, shared_blocks=1)
    q = make_q(3, 24, c.row, 6)
    _, lse = run_decode(c, q, [2, 0, 1], 1, 24, 0.07)
    w = torch.zeros(3, 40 * 64, device=DEV)
    run_weights(c, q, [2, 0, 1], 1, 24, 0.07, lse, 1.0, w)
    assert c.bits() == 0
    # 2^-11 from the terms (as above) and from lse each
    assert bool(((w.double().sum(1) - 24).abs() <= 24 * 2.0 ** -10).all())
    for s, n in enumerate(lens):
        assert bool((w[s, n:] == 0).all())


@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_scales(scale):
    c = Paged(20, 32, 256, 32, 2, 8)
    rows = c.fill([150, 40], seed=95)
    q = make_q(4, 5, c.row, 96)
    lse = lse64(rows, q, [0, 1], 2, 5, scale)
    old = torch.zeros(2, 256, device=DEV)
    got = run_weights(c, q, [0, 1], 2, 5, scale, lse, 1.0, old.clone())
    assert c.bits() == 0
    check(rows, q, [0, 1], 2, 5, scale, lse, 1.0, old, got)


def test_more_than_512_sequences_and_layers():
    lens = [(i * 37) % 150 for i in range(600)]
    c = Paged(2 + sum(-(-n // 32) for n in lens), 32, 128, 16, 600, 5, layers=3)
    rows = c.fill(lens, seed=60, layer=2)
    q = make_q(600, 5, c.row, 61)
    seqs = list(range(600))
    lse = lse64(rows, q, seqs, 1, 5, 0.1)
    old = torch.rand(600, 160, device=DEV)
    got = run_weights(c, q, seqs, 1, 5, 0.1, lse, 1.0, old.clone(), layer=2)
    assert c.bits() == 0
    check(rows, q, seqs, 1, 5, 0.1, lse, 1.0, old, got)


def test_refused_on_the_device():
    c = Paged(20, 64, 512, 64, 4, 6)
    rows = c.fill([100, 200, 30], seed=40)
    q = make_q(5, 16, c.row, 41)
    seqs = [0, 9, 2, 0, -1]
    lse = lse64(rows, q, [0, 0, 2, 0, 0], 1, 16, 0.07)
    old = torch.rand(4, 384, device=DEV)
    got = run_weights(c, q, seqs, 1, 16, 0.07, lse, 1.0, old.clone())
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    check(rows, q[:1], [0], 1, 16, 0.07, lse[:1], 1.0, torch.cat([old[:2], got[2:]]), got)     # the first entry of 0 alone
    check(rows, q[2:3], [2], 1, 16, 0.07, lse[2:3], 1.0, torch.cat([got[:2], old[2:]]), got)
    c.table[1, 2] = -1
    got = run_weights(c, q[:2], [0, 1], 1, 16, 0.07, lse[:2], 1.0, old.clone())
    assert c.bits() == moe.MOE_DEV_ERR_BAD_PAGE
    assert torch.equal(got[2:], old[2:])
    check(rows, q[:1], [0], 1, 16, 0.07, lse[:1], 1.0, old, torch.cat([got[:1], old[1:]]))


def test_a_repeat_far_down_the_list():
    """The repeat lies in another launch's share of the sequences."""
    c = Paged(4, 16, 128, 16, 600, 1)
    rows = c.fill([16], seed=3)
    q = make_q(600, 2, c.row, 4)
    lse = lse64(rows, q[:1], [0], 1, 2, 0.1).repeat(600, 1)
    old = torch.zeros(600, 16, device=DEV)
    got = run_weights(c, q, [0] + list(range(1, 599)) + [0], 1, 2, 0.1, lse, 1.0, old.clone())
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    check(rows, q[:1], [0], 1, 2, 0.1, lse[:1], 1.0, old, got)


def test_bad_values_touch_their_own_token():
    c = Paged(12, 32, 256, 32, 2, 6)
    rows = c.fill([100, 129], seed=100)
    q = make_q(6, 5, c.row, 101)
    lse = lse64(rows, q, [0, 1], 3, 5, 0.1)
    old = torch.zeros(2, 192, device=DEV)
    clean = run_weights(c, q, [0, 1], 3, 5, 0.1, lse, 1.0, old.clone())
    c.pages[0, int(c.table[0, 1]), 3, 7] = float("nan")
    got = run_weights(c, q, [0, 1], 3, 5, 0.1, lse, 1.0, old.clone())
    assert c.bits() == 0 and bool(torch.isnan(got[0, 35]))
    got[0, 35] = clean[0, 35]
    assert torch.equal(got, clean)


def test_queries_behind_the_lists_last_are_not_read():
    """Rows of q and lse past the call's own hold NaN."""
    c = Paged(12, 32, 256, 32, 1, 6)
    rows = c.fill([100], seed=100)
    q, lse = make_q(4, 5, c.row, 101), torch.full((4, 5), float("nan"), device=DEV)
    lse[:1] = lse64(rows, q, [0], 1, 5, 0.1)
    q[1:] = float("nan")
    old = torch.zeros(1, 192, device=DEV)
    got = run_weights(c, q, [0], 1, 5, 0.1, lse, 1.0, old.clone())
    assert c.bits() == 0
    check(rows, q[:1], [0], 1, 5, 0.1, lse[:1], 1.0, old, got)


def test_in_a_graph_on_another_stream():
    c = Paged(40, 16, 512, 64, 2, 12)
    rows = c.fill([60, 110], seed=70)
    q = make_q(2, 16, c.row, 71)
    seqs, w = i32([1, 0]), torch.zeros(2, 192, device=DEV)
    n = moe.moe_latent_weights_workspace_size(c.handle, 2, 1, 16)
    ws, lse = torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV), torch.zeros(2, 16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_latent_weights(c.handle, 0, q, seqs, 2, 1, 16, 0.07, lse, 0.5, w, ws, ws.numel(), c.status)
    for now in ([60, 110], [31, 100]):
        cut = [x[:k] for x, k in zip(rows, now)]
        c.lens.copy_(i32(now))
        lse.copy_(lse64(cut, q, [1, 0], 1, 16, 0.07))
        old = w.clone()
        g.replay()
        torch.cuda.synchronize()
        check(cut, q, [1, 0], 1, 16, 0.07, lse, 0.5, old, w)
    assert c.bits() == 0
