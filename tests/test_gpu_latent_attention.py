"""Latent attention over the paged cache (absorbed, shared prefix, expanded)
against the definition in 64 bits, on caches whose unused places hold NaN.

Bounds, from the roundings the header states (u = 2^-8, the unit roundoff of
bf16's 8 significand bits: 1 + 2^-8 rounds to 1):
* absorbed: the probabilities are rounded to bf16 (each off by at most u of
  itself), the output once more, everything else is fp32: scores of a few
  hundred products carry about 2^-24 * sqrt(576) * sum|q||k| scale < 2^-14, which
  2^-11 covers four times over at the spreads used here.  So
  |err| <= u |ref| + (u + 2^-11) sum p|v|, elementwise.
* expanded: k and v are rounded too.  v adds u sum p|v|; k moves a score by at
  most e = u * scale * sum|q||k|, and a probability by at most exp(2e) - 1.
  Independent roundings have far smaller norms: each source is 2^-9 / sqrt(3)
  of its operand's norm or less, four of them 2.3e-3 together; the Frobenius
  bound is 4e-3.
* lse is fp32: 2^-14 absolute from the scores, on values of order 10.
"""
import math

import pytest
import torch

import edge_moe_serving_gb300 as moe
from kv_helpers import DEV, Paged, attend64

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
LSE_TOL = 2.0 ** -11


def run_decode(c, q, seqs, Q, heads, scale, shared=0, lse=True, stream=None, layer=0):
    B = len(seqs)
    n = moe.moe_latent_decode_workspace_size(c.handle, B, Q, heads, shared)
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device=DEV)      # NaN wherever something reads it unwritten
    out = torch.full((B * Q, heads, c.rank), float("nan"), dtype=torch.bfloat16, device=DEV)
    l = torch.full((B * Q, heads), float("nan"), device=DEV) if lse else None
    moe.moe_latent_decode(c.handle, layer, q, torch.tensor(seqs, dtype=torch.int32, device=DEV), B, Q, heads, scale,
                          shared, out, l, ws, ws.numel(), c.status, stream)
    return out, l


def check_decode(c, rows, q, seqs, Q, heads, scale, out, lse):
    for b, s in enumerate(seqs):
        x = rows[s]
        qb = q[b * Q:(b + 1) * Q].cpu().double().reshape(Q * heads, -1)
        limit = [len(x) - Q + i + 1 for i in range(Q) for _ in range(heads)]
        ref, mag, ref_lse = attend64(qb, x, x[:, :c.rank], scale, limit)
        got = out[b * Q:(b + 1) * Q].cpu().double().reshape(Q * heads, -1)
        bound = U * ref.abs() + (U + 2.0 ** -11) * mag + 1e-30
        bad = (got - ref).abs() > bound
        assert not bool(bad.any()) and bool(torch.isfinite(got).all()), (b, s, int(bad.sum()), float(((got - ref).abs() / bound).max()))
        if lse is not None:
            g = lse[b * Q:(b + 1) * Q].cpu().double().reshape(-1)
            none = ref_lse == -math.inf
            assert bool((g[none] == -math.inf).all())
            assert bool(((g - ref_lse)[~none].abs() <= LSE_TOL).all()), float((g - ref_lse)[~none].abs().max())


def make_q(n, heads, row, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, row, generator=g) * spread).to(torch.bfloat16).to(DEV)


DECODE = [
    # rank, rope, page, heads, Q, lens
    (512, 64, 64, 16, 1, [1]),
    (512, 64, 64, 128, 1, [63, 64, 65, 127, 128, 129]),
    (512, 64, 16, 64, 1, [1, 2, 15, 16, 17, 700, 333, 64]),
    (512, 64, 128, 20, 1, [300, 1, 129, 128, 1000]),
    (512, 64, 32, 8, 2, [2, 33, 95, 1]),              # a sequence shorter than Q: its first query sees nothing
    (256, 32, 64, 48, 3, [5, 200, 64, 3]),
    (128, 0, 16, 1, 1, [1, 40, 16]),
    (384, 16, 32, 37, 4, [77, 4, 400]),
    (512, 64, 64, 128, 8, [8, 150, 1029]),
    (256, 48, 128, 7, 1, [0, 5, 0, 130]),             # empty sequences
    (512, 64, 64, 96, 1, [2000, 3, 511]),
    (512, 64, 64, 72, 2, [640, 65]),
]


@pytest.mark.parametrize("rank,rope,page,heads,Q,lens", DECODE)
def test_decode(rank, rope, page, heads, Q, lens):
    blocks = [-(-n // page) for n in lens]
    c = Paged(sum(blocks) + 5, page, rank, rope, len(lens) + 2, max(blocks) + 1)
    rows = c.fill(lens, seed=heads)
    q = make_q(len(lens) * Q, heads, c.row, 3)
    scale = 1.0 / math.sqrt(128 + rope)
    seqs = list(range(len(lens)))[::-1]
    out, lse = run_decode(c, q, seqs, Q, heads, scale)
    assert c.bits() == 0
    check_decode(c, rows, q, seqs, Q, heads, scale, out, lse)
    again, _ = run_decode(c, q, seqs, Q, heads, scale, lse=False)
    assert torch.equal(out, again)                    # same bits on every run, lse asked for or not


PREFIX = [
    # rank, rope, page, heads, Q, shared blocks, own tokens
    (512, 64, 32, 16, 1, 32, [1, 200, 33, 64, 65, 7, 128, 90]),
    (512, 64, 64, 64, 1, 5, [70, 1, 130]),
    (512, 64, 16, 8, 2, 3, [2, 17, 16, 40, 100]),      # a prefix that ends inside a tile
    (256, 32, 128, 20, 1, 9, [1, 5, 300]),
    (512, 64, 64, 128, 2, 4, [2, 65]),
    (128, 64, 16, 12, 1, 65, [0, 3, 0, 50]),           # nothing after the prefix
    (512, 64, 64, 32, 1, 40, [10] * 33),
]


@pytest.mark.parametrize("rank,rope,page,heads,Q,shared_blocks,own", PREFIX)
def test_shared_prefix(rank, rope, page, heads, Q, shared_blocks, own):
    shared = shared_blocks * page
    lens = [shared + n for n in own]
    blocks = [-(-n // page) for n in lens]
    c = Paged(sum(blocks) + 5, page, rank, rope, len(lens), max(blocks))
    rows = c.fill(lens, seed=heads, shared_blocks=shared_blocks)
    q = make_q(len(lens) * Q, heads, c.row, 4)
    scale = 1.0 / math.sqrt(128 + rope)
    seqs = list(range(len(lens)))
    out, lse = run_decode(c, q, seqs, Q, heads, scale, shared=shared)
    assert c.bits() == 0
    check_decode(c, rows, q, seqs, Q, heads, scale, out, lse)


def test_decode_prefix_longer_than_a_sequence():
    """A sequence inside the shared tokens sees its own length of them."""
    c = Paged(40, 16, 512, 64, 3, 12)
    rows = c.fill([100, 160, 70], seed=1, shared_blocks=6)
    q = make_q(3, 16, c.row, 5)
    out, lse = run_decode(c, q, [0, 1, 2], 1, 16, 0.07, shared=96)
    assert c.bits() == 0
    check_decode(c, rows, q, [0, 1, 2], 1, 16, 0.07, out, lse)


@pytest.mark.parametrize("scale,spread", [(-0.07, 1.0), (0.0, 1.0), (0.07, 8.0)])
def test_decode_score_ranges(scale, spread):
    """Negative and zero scales, and scores of hundreds that grow along the sequence (every rescaling is met).
    Scores of that size carry an error of 2^-24 * their magnitude * a few: spread 8 raises the sum of |q||k| scale to
    about 1700, and 2^-24 * sqrt(576) * 1700 = 2.4e-3 of relative error in a probability is covered by the bound below."""
    c = Paged(60, 64, 512, 64, 2, 24)
    lens = [1500, 200]
    rows = c.fill(lens, seed=2)
    for s in range(2):                                 # rows grow in size along the sequence
        n = lens[s]
        ramp = torch.linspace(0.02, spread, n)[:, None].double()
        rows[s] = (rows[s] * ramp).to(torch.bfloat16).double()
        for b in range(-(-n // 64)):
            part = rows[s][b * 64:(b + 1) * 64]
            c.pages[0, int(c.table[s, b]), :len(part)] = part.to(torch.bfloat16).to(DEV)
    q = make_q(2, 32, c.row, 6, spread=spread)
    out, lse = run_decode(c, q, [0, 1], 1, 32, scale)
    assert c.bits() == 0
    for b in range(2):
        x = rows[b]
        ref, mag, ref_lse = attend64(q[b].cpu().double(), x, x[:, :512], scale, [lens[b]] * 32)
        got = out[b].cpu().double()
        slack = 2 * 2.4e-3 if spread > 1 else 2.0 ** -11
        assert bool(((got - ref).abs() <= U * ref.abs() + (U + slack) * mag + 1e-30).all())
        assert bool(((lse[b].cpu().double() - ref_lse).abs() <= (4e-3 if spread > 1 else LSE_TOL)).all())


def test_decode_infinite_and_nan_rows():
    """NaN in a row a query sees reaches that query's outputs and no other sequence's; an infinite negative score
    leaves its token out."""
    c = Paged(20, 16, 512, 64, 3, 6)
    rows = c.fill([50, 50, 50], seed=3)
    c.pages[0, int(c.table[1, 2]), 3] = float("nan")
    q = make_q(3, 16, c.row, 7)
    out, _ = run_decode(c, q, [0, 1, 2], 1, 16, 0.07)
    assert bool(torch.isnan(out[1]).all())
    check_decode(c, rows, q[0:1], [0], 1, 16, 0.07, out[0:1], None)
    check_decode(c, rows, q[2:3], [2], 1, 16, 0.07, out[2:3], None)
    # the rotary part alone decides the score: -inf for one token, whose latent is finite
    rows = c.fill([50, 50, 50], seed=4)
    q2 = q.clone()
    q2[:, :, 512:] = 0
    q2[:, :, 512] = 1.0
    for s in range(3):
        rows[s][7, 512] = -3e38                        # -3e38 * scale * log2(e) leaves fp32 for scale 4
        c.pages[0, int(c.table[s, 0]), 7, 512] = -3e38
    q2[:, :, :512] = 0
    out, lse = run_decode(c, q2, [0, 1, 2], 1, 16, 4.0)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for b in range(3):
        keep = [t for t in range(50) if t != 7]
        x = rows[b][keep]
        ref, mag, _ = attend64(q2[b].cpu().double(), x, x[:, :512], 4.0, [49] * 16)
        assert bool(((out[b].cpu().double() - ref).abs() <= U * ref.abs() + (U + 2.0 ** -11) * mag).all())


def test_decode_layers_streams_and_bad_entries():
    c = Paged(30, 32, 512, 64, 4, 6, layers=3)
    rows = c.fill([100, 40, 33, 0], seed=8, layer=2)
    q = make_q(4, 16, c.row, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = run_decode(c, q, [0, 1, 2, 3], 1, 16, 0.07, layer=2)
    s.synchronize()
    assert c.bits() == 0
    check_decode(c, rows, q, [0, 1, 2, 3], 1, 16, 0.07, out, lse)
    out, lse = run_decode(c, q, [0, 99, -1, 2], 1, 16, 0.07, layer=2)     # ids out of range: zeros
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    assert bool((out[1:3] == 0).all()) and bool((lse[1:3] == -math.inf).all())
    check_decode(c, rows, q[0:1], [0], 1, 16, 0.07, out[0:1], lse[0:1])
    check_decode(c, rows, q[3:4], [2], 1, 16, 0.07, out[3:4], lse[3:4])
    c.table[1, 1] = 30                                                     # a page past the pool
    c.table[2, 0] = -1
    out, lse = run_decode(c, q, [0, 1, 2, 3], 1, 16, 0.07, layer=2)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_PAGE
    check_decode(c, rows, q[0:1], [0], 1, 16, 0.07, out[0:1], lse[0:1])
    out, lse = run_decode(c, q, [0, 1, 0, 3], 1, 16, 0.07, layer=2)        # one sequence twice in a batch
    assert torch.equal(out[0].isnan(), out[2].isnan())


def test_decode_long_ragged_batch():
    """Work split over every SM: one long sequence among short and empty ones, and one alone."""
    lens = [9000, 1, 0, 4097, 77, 2048, 640]
    c = Paged(sum(-(-n // 64) for n in lens) + 1, 64, 512, 64, len(lens), 150)
    rows = c.fill(lens, seed=9)
    for heads, seqs in ((64, list(range(7))), (128, [0]), (16, [3, 0, 2]), (8, [0])):
        q = make_q(len(seqs), heads, c.row, heads)
        out, lse = run_decode(c, q, seqs, 1, heads, 0.07)
        assert c.bits() == 0
        check_decode(c, rows, q, seqs, 1, heads, 0.07, out, lse)


def test_decode_padded_batch():
    """A batch of fixed size whose unused slots are -1, with more query rows than SMs, in a workspace of exactly the
    size asked for: zeros and -infinity for the padding and for empty sequences, also in front of the others."""
    c = Paged(40, 32, 512, 64, 6, 12)
    rows = c.fill([0, 300, 64, 0, 17], seed=10)
    for seqs in ([-1, -1, 0, 1, 2, 3, 4, -1], [-1] * 8, [0, 3, 0], [1, -1, 2, 99, -1, -1, -1, -1]):
        q = make_q(len(seqs), 64, c.row, 11)
        out, lse = run_decode(c, q, seqs, 1, 64, 0.07)
        assert c.bits() == (0 if seqs == [0, 3, 0] else moe.MOE_DEV_ERR_BAD_SEQ)
        for b, s in enumerate(seqs):
            if not 0 <= s < 6 or not len(rows[s]):
                assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            else:
                check_decode(c, rows, q[b:b + 1], [s], 1, 64, 0.07, out[b:b + 1], lse[b:b + 1])


# ------------------------------------------------------------------ expanded form
def run_prefill(c, q, seqs, offsets, heads, dn, dv, w, scale, kv_tokens, layer=0):
    B, T = len(seqs), q.shape[0]
    n = moe.moe_latent_prefill_workspace_size(c.handle, B, T, heads, dn, dv, kv_tokens)
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((T, heads, dv), float("nan"), dtype=torch.bfloat16, device=DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    moe.moe_latent_prefill(c.handle, layer, q, i32(seqs), i32(offsets), B, T, heads, dn, dv, w, scale, kv_tokens, out,
                           ws, ws.numel(), c.status)
    return out


def check_prefill(c, rows, q, seqs, offsets, heads, dn, w, scale, out):
    err = ref_sq = 0.0
    for b, s in enumerate(seqs):
        n = offsets[b + 1] - offsets[b]
        x = rows[s]
        limit = [len(x) - n + j + 1 for j in range(n)]
        for h in range(heads):
            wh = w[h].cpu().double()
            k = torch.cat([x[:, :c.rank] @ wh[:dn].T, x[:, c.rank:]], 1)
            v = x[:, :c.rank] @ wh[dn:].T
            qh = q[offsets[b]:offsets[b + 1], h].cpu().double()
            ref, mag, _ = attend64(qh, k, v, scale, limit)
            got = out[offsets[b]:offsets[b + 1], h].cpu().double()
            assert bool(torch.isfinite(got).all()), (b, h)
            if n == 0:
                continue
            e = U * abs(scale) * (qh.abs() @ k.abs().T).amax(1, keepdim=True)
            bound = U * ref.abs() + (2 * U + 2.0 ** -11 + torch.expm1(2 * e)) * mag
            assert not bool(((got - ref).abs() > bound).any()), (b, h, float(((got - ref).abs() / bound).max()))
            err += float((got - ref).square().sum())
            ref_sq += float(ref.square().sum())
    assert math.sqrt(err) <= 4e-3 * math.sqrt(ref_sq), math.sqrt(err / ref_sq)


def make_w(heads, feats, rank, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(heads, feats, rank, generator=g) / math.sqrt(rank)).to(torch.bfloat16).to(DEV)


PREFILL = [
    # rank, rope, page, heads, dn, dv, lens, new
    (512, 64, 64, 2, 128, 128, [1], [1]),
    (512, 64, 16, 3, 128, 128, [300, 1, 129, 128, 64], [300, 1, 129, 128, 64]),
    (512, 64, 64, 1, 128, 128, [700, 257], [130, 1]),          # chunks over what is cached
    (256, 32, 32, 2, 64, 128, [200, 77], [200, 33]),
    (128, 0, 128, 1, 128, 64, [333], [333]),
    (384, 16, 16, 2, 64, 64, [90, 5, 260], [17, 5, 259]),
    (512, 64, 64, 1, 128, 128, [1025], [1025]),
    (512, 48, 128, 5, 128, 128, [127, 0, 255], [127, 0, 2]),   # a sequence without tokens
]


@pytest.mark.parametrize("rank,rope,page,heads,dn,dv,lens,new", PREFILL)
def test_prefill(rank, rope, page, heads, dn, dv, lens, new):
    blocks = [-(-n // page) for n in lens]
    c = Paged(sum(blocks) + 3, page, rank, rope, len(lens), max(blocks) + 1, layers=2)
    rows = c.fill(lens, seed=heads + 20, layer=1)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    q = make_q(offsets[-1], heads, dn + rope, 21)
    w = make_w(heads, dn + dv, rank, 22)
    scale = 1.0 / math.sqrt(dn + rope)
    seqs = list(range(len(lens)))
    out = run_prefill(c, q, seqs, offsets, heads, dn, dv, w, scale, sum(lens), layer=1)
    assert c.bits() == 0
    check_prefill(c, rows, q, seqs, offsets, heads, dn, w, scale, out)
    assert torch.equal(out, run_prefill(c, q, seqs, offsets, heads, dn, dv, w, scale, sum(lens) + 500, layer=1))


def test_prefill_growing_scores():
    """Scores that grow along the keys, so that the running maximum rises in every tile."""
    c = Paged(12, 64, 512, 64, 1, 12)
    rows = c.fill([600], seed=30)
    ramp = torch.linspace(0.1, 6.0, 600)[:, None].double()
    rows[0][:, 512:] = (rows[0][:, 512:].abs() * ramp).to(torch.bfloat16).double()
    for b in range(10):
        part = rows[0][b * 64:(b + 1) * 64]
        c.pages[0, int(c.table[0, b]), :len(part)] = part.to(torch.bfloat16).to(DEV)
    q = make_q(600, 2, 192, 31)
    q[:, :, 128:] = q[:, :, 128:].abs()
    w = make_w(2, 256, 512, 32)
    scale = 1.0 / math.sqrt(192)
    out = run_prefill(c, q, [0], [0, 600], 2, 128, 128, w, scale, 600)
    check_prefill(c, rows, q, [0], [0, 600], 2, 128, w, scale, out)


def test_prefill_refused_on_the_device():
    c = Paged(20, 64, 512, 64, 4, 6)
    rows = c.fill([100, 200, 30], seed=40)
    q = make_q(60, 2, 192, 41)
    w = make_w(2, 256, 512, 42)
    out = run_prefill(c, q, [0, 1], [0, 20, 60], 2, 128, 128, w, 0.07, 20)        # 300 tokens, room for far fewer
    assert c.bits() == moe.MOE_DEV_ERR_CAPACITY
    assert bool(torch.isnan(out).all())
    out = run_prefill(c, q, [0, 9], [0, 20, 60], 2, 128, 128, w, 0.07, 300)       # a bad id
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    check_prefill(c, rows, q[:20], [0], [0, 20], 2, 128, w, 0.07, out[:20])
    assert bool(torch.isnan(out[20:]).all())
    out = run_prefill(c, q, [2, 1], [0, 40, 60], 2, 128, 128, w, 0.07, 300)       # more queries than tokens
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    assert bool(torch.isnan(out[:40]).all())
    check_prefill(c, rows, q[40:], [1], [0, 20], 2, 128, w, 0.07, out[40:])
    c.table[1, 3] = -1
    out = run_prefill(c, q, [0, 1], [0, 20, 60], 2, 128, 128, w, 0.07, 300)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_PAGE
    check_prefill(c, rows, q[:20], [0], [0, 20], 2, 128, w, 0.07, out[:20])


def test_both_forms_agree():
    """One new token through the expanded form equals the absorbed form with the projections folded in by hand."""
    c = Paged(30, 64, 512, 64, 2, 12)
    c.fill([500, 260], seed=50)
    heads, scale = 4, 1.0 / math.sqrt(192)
    q = make_q(2, heads, 192, 51)
    w = make_w(heads, 256, 512, 52)
    out = run_prefill(c, q, [0, 1], [0, 1, 2], heads, 128, 128, w, scale, 760).double()
    ql = torch.einsum("bhd,hdr->bhr", q[..., :128].double(), w[:, :128].double())
    qa = torch.cat([ql, q[..., 128:].double()], -1).to(torch.bfloat16)
    lat, _ = run_decode(c, qa, [0, 1], 1, heads, scale)
    other = torch.einsum("bhr,hdr->bhd", lat.double(), w[:, 128:].double())
    assert c.bits() == 0
    # the absorbed query is rounded to bf16, as k is in the other form: each within the expanded form's 4e-3
    assert float((out - other).norm() / out.norm()) <= 8e-3


@pytest.mark.parametrize("B,heads", [(3, 16), (40, 8), (530, 5)])
def test_shared_prefix_of_a_bad_id(B, heads):
    """The shared tokens are the first sequence's: where its id is outside the cache no row gets another's tokens."""
    c = Paged(300, 16, 128, 16, 4, 12)
    c.pages[0, 0] = 1.0                                    # what a stand-in for the missing table would name
    rows = c.fill([100, 160, 70, 33], seed=62, shared_blocks=2)
    q = make_q(B, heads, c.row, 63)
    for first in (-1, 4):
        out, lse = run_decode(c, q, [first] + [i % 4 for i in range(1, B)], 1, heads, 0.1, shared=32)
        assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    seqs = [0] + [-1 if i % 5 == 2 else i % 4 for i in range(1, B)]      # elsewhere a bad id is that row's alone
    out, lse = run_decode(c, q, seqs, 1, heads, 0.1, shared=32)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    for b in (0, 1, 2, B - 1):
        if seqs[b] < 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
        else:
            check_decode(c, rows, q[b:b + 1], [seqs[b]], 1, heads, 0.1, out[b:b + 1], lse[b:b + 1])


def test_more_than_one_launch_of_sequences():
    """More sequences than one launch takes (512), with and without a shared prefix."""
    lens = [64 + (i * 7) % 40 for i in range(530)]
    c = Paged(2 + sum(-(-n // 32) for n in lens), 32, 128, 16, 530, 4)
    rows = c.fill(lens, seed=60, shared_blocks=2)
    q = make_q(530, 5, c.row, 61)
    for shared in (0, 64):
        out, lse = run_decode(c, q, list(range(530)), 1, 5, 0.1, shared=shared)
        assert c.bits() == 0
        for b in (0, 1, 511, 512, 513, 529):
            check_decode(c, rows, q[b:b + 1], [b], 1, 5, 0.1, out[b:b + 1], lse[b:b + 1])


def test_attention_in_a_graph():
    """Both calls captured once and replayed after the cache has grown: lengths and tables are read on the device."""
    c = Paged(40, 16, 512, 64, 2, 12)
    lens = [40, 90]
    rows = c.fill([60, 110], seed=70)
    q = make_q(2, 16, c.row, 71)
    qp, w = make_q(2, 2, 192, 72), make_w(2, 256, 512, 73)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    seqs, offsets = i32([0, 1]), i32([0, 1, 2])
    n1 = moe.moe_latent_decode_workspace_size(c.handle, 2, 1, 16, 0)
    n2 = moe.moe_latent_prefill_workspace_size(c.handle, 2, 2, 2, 128, 128, 200)
    ws1, ws2 = (torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (n1, n2))
    out = torch.zeros(2, 16, 512, dtype=torch.bfloat16, device=DEV)
    outp = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    c.lens.copy_(i32(lens))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def both():
        moe.moe_latent_decode(c.handle, 0, q, seqs, 2, 1, 16, 0.07, 0, out, None, ws1, n1, c.status)
        moe.moe_latent_prefill(c.handle, 0, qp, seqs, offsets, 2, 2, 2, 128, 128, w, 0.07, 200, outp, ws2, n2, c.status)

    with torch.cuda.stream(s):
        both()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both()
    for now in (lens, [60, 110]):
        c.lens.copy_(i32(now))
        g.replay()
        torch.cuda.synchronize()
        cut = [x[:n] for x, n in zip(rows, now)]
        check_decode(c, cut, q, [0, 1], 1, 16, 0.07, out, None)
        check_prefill(c, cut, qp, [0, 1], [0, 1, 2], 2, 128, w, 0.07, outp)
    assert c.bits() == 0


def test_prefill_values_beyond_the_f16_range():
    """A value past 65504 is clamped and reported; keys of that size are not touched (they stay bf16)."""
    c = Paged(4, 64, 128, 16, 1, 3)
    c.fill([80], seed=80)
    w = make_w(1, 256, 128, 81)
    q = torch.zeros(1, 1, 144, dtype=torch.bfloat16, device=DEV)
    w[:, :128] *= 1e6
    run_prefill(c, q, [0], [0, 1], 1, 128, 128, w, 0.1, 80)
    assert c.bits() == 0
    w[:, 128:] *= 1e6
    out = run_prefill(c, q, [0], [0, 1], 1, 128, 128, w, 0.1, 80)
    assert c.bits() == moe.MOE_DEV_ERR_RANGE
    assert bool(torch.isfinite(out).all()) and float(out.abs().max()) <= 65536.0


@pytest.mark.parametrize("heads,new,cached", [(3, 70, 5000), (2, 300, 1500)])
def test_prefill_token_shares(heads, new, cached):
    """Few query blocks over many tokens: their tokens are shared out and the shares joined."""
    n = cached + new
    c = Paged(-(-n // 64) + 1, 64, 512, 64, 1, -(-n // 64))
    rows = c.fill([n], seed=90)
    q, w = make_q(new, heads, 192, 91), make_w(heads, 256, 512, 92)
    out = run_prefill(c, q, [0], [0, new], heads, 128, 128, w, 192 ** -0.5, n)
    assert c.bits() == 0
    check_prefill(c, rows, q, [0], [0, new], heads, 128, w, 192 ** -0.5, out)
    assert torch.equal(out, run_prefill(c, q, [0], [0, new], heads, 128, 128, w, 192 ** -0.5, n))


@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_prefill_scales(scale):
    c = Paged(8, 32, 256, 32, 2, 8)
    rows = c.fill([150, 40], seed=95)
    q, w = make_q(60, 2, 96, 96), make_w(2, 128, 256, 97)
    out = run_prefill(c, q, [0, 1], [0, 40, 60], 2, 64, 64, w, scale, 190)
    assert c.bits() == 0
    check_prefill(c, rows, q, [0, 1], [0, 40, 60], 2, 64, w, scale, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_values_reach_only_the_rows_that_see_them(bad):
    """A token's NaN or infinite latent: queries before it are what they would be without it."""
    Q, heads = 3, 5
    c = Paged(12, 32, 256, 32, 2, 6)
    rows = c.fill([100, 129], seed=100)
    q, qp, w = make_q(2 * Q, heads, c.row, 101), make_q(60, 2, 96, 102), make_w(2, 128, 256, 103)
    clean = [x.clone() for x in rows]
    for s, n in ((0, 100), (1, 129)):          # the last token of each sequence
        page = int(c.table[s, (n - 1) // 32])
        c.pages[0, page, (n - 1) % 32, 7] = bad
        clean[s][n - 1, 7] = 0.0
    out, _ = run_decode(c, q, [0, 1], Q, heads, 0.1)
    seen = torch.arange(2 * Q, device=DEV) % Q == Q - 1
    assert c.bits() == 0 and bool(torch.isfinite(out[~seen]).all())
    for b, n in ((0, 100), (1, 129)):
        for i in range(Q - 1):
            at = b * Q + i
            check_decode(c, {b: clean[b][:n - Q + i + 1]}, q[at:at + 1], [b], 1, heads, 0.1, out[at:at + 1], None)
    outp = run_prefill(c, qp, [0, 1], [0, 30, 60], 2, 64, 64, w, 0.1, 229)
    c.bits()                                   # an infinite value is beyond the f16 range: reported
    keep = [i for i in range(60) if i % 30 != 29]
    assert bool(torch.isfinite(outp[keep]).all())
    for b, n in ((0, 100), (1, 129)):
        check_prefill(c, {b: clean[b][:n - 1]}, qp[30 * b:30 * b + 29], [b], [0, 29], 2, 64, w, 0.1,
                      outp[30 * b:30 * b + 29])
    if bad != bad:
        assert bool(torch.isnan(out[seen]).any()) and bool(torch.isnan(outp[[29, 59]]).any())


@pytest.mark.parametrize("B", [32, 33, 70])
def test_prefill_of_many_sequences(B):
    """Around and past the 32 sequences whose plan needs no launch of its own; some without queries, some empty."""
    lens = [0 if i % 9 == 4 else 1 + (37 * i) % 200 for i in range(B)]
    new = [0 if i % 5 == 3 else min(n, 1 + (11 * i) % 60) for i, n in enumerate(lens)]
    c = Paged(sum(-(-n // 16) for n in lens) + 3, 16, 128, 16, B, 14)
    rows = c.fill(lens, seed=B)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    q, w = make_q(offsets[-1], 3, 80, 104), make_w(3, 128, 128, 105)
    out = run_prefill(c, q, list(range(B)), offsets, 3, 64, 64, w, 0.12, sum(lens))
    assert c.bits() == 0
    some = [b for b in range(B) if new[b]]
    check_prefill(c, rows, q, some, [offsets[b] for b in some] + [offsets[-1]], 3, 64, w, 0.12, out)
    # no room for the lengths: reported, nothing written
    run_prefill(c, q, list(range(B)), offsets, 3, 64, 64, w, 0.12, 1)
    assert c.bits() == (moe.MOE_DEV_ERR_CAPACITY if sum(-(-n // 128) for n in lens) > B else 0)


WIDTHS = [
    # rank, rope, page, heads, dn, dv, lens, new: the widths of keys and values that PREFILL leaves out
    (512, 0, 64, 3, 64, 64, [300, 1, 129], [300, 1, 129]),
    (256, 0, 32, 2, 64, 128, [257, 600], [257, 31]),
    (512, 64, 16, 3, 128, 64, [130, 520, 77], [130, 400, 76]),
    (128, 0, 128, 2, 128, 128, [513], [513]),
    (512, 64, 64, 2, 64, 64, [1000], [260]),
]


@pytest.mark.parametrize("rank,rope,page,heads,dn,dv,lens,new", WIDTHS)
def test_prefill_widths(rank, rope, page, heads, dn, dv, lens, new):
    """Every pair of widths, with and without a rotary part, whole prompts and chunks that are shared out."""
    test_prefill(rank, rope, page, heads, dn, dv, lens, new)


@pytest.mark.parametrize("rope,dn,dv", [(0, 64, 64), (0, 64, 128), (32, 128, 64), (0, 128, 128)])
def test_prefill_widths_in_token_shares(rope, dn, dv):
    c = Paged(40, 128, 256, rope, 1, 40)
    rows = c.fill([4900], seed=110)
    q, w = make_q(40, 2, dn + rope, 111), make_w(2, dn + dv, 256, 112)
    out = run_prefill(c, q, [0], [0, 40], 2, dn, dv, w, 0.09, 4900)
    assert c.bits() == 0
    check_prefill(c, rows, q, [0], [0, 40], 2, dn, w, 0.09, out)


def test_one_workspace_for_all_chunks():
    """The workspace of a full chunk takes the short last chunk, that of a large fan-out a smaller one: same results as
    with a workspace of their own."""
    c = Paged(60, 64, 512, 64, 5, 40)
    rows = c.fill([2303, 320, 330, 340, 350], seed=120, shared_blocks=4)
    heads, scale = 2, 192 ** -0.5
    q, w = make_q(1280, heads, 192, 121), make_w(heads, 256, 512, 122)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    n = moe.moe_latent_prefill_workspace_size(c.handle, 1, 1280, heads, 128, 128, 2303)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    for T in (1280, 255, 1):
        own = run_prefill(c, q[:T], [0], [0, T], heads, 128, 128, w, scale, 2303)
        out = torch.full((T, heads, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        moe.moe_latent_prefill(c.handle, 0, q, i32([0]), i32([0, T]), 1, T, heads, 128, 128, w, scale, 2303, out, ws, n,
                               c.status)
        assert c.bits() == 0 and torch.equal(out, own)
        check_prefill(c, rows, q[:T], [0], [0, T], heads, 128, w, scale, out)
    q = make_q(5, 16, c.row, 123)
    n = moe.moe_latent_decode_workspace_size(c.handle, 5, 1, 16, 256)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    for B in (5, 4, 1):
        seqs = list(range(B))
        own, _ = run_decode(c, q[:B], seqs, 1, 16, scale, shared=256)
        out = torch.full((B, 16, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
        moe.moe_latent_decode(c.handle, 0, q, i32(seqs), B, 1, 16, scale, 256, out, None, ws, n, c.status)
        assert c.bits() == 0 and torch.equal(out, own)
        check_decode(c, rows, q[:B], seqs, 1, 16, scale, out, None)


@pytest.mark.parametrize("heads,n,bits", [(1, 5000, 26.5), (160, 900, 26.5), (160, 900, 20.5), (1, 5000, 31.0)])
def test_prefill_long_tail_behind_one_token(heads, n, bits):
    """The first token takes nearly all the probability and has value 0; the output is the tail's, n - 1 tokens of
    probability 2^-bits each.  Scores come from the rotary part alone, which is not rounded, and all values are 0 or 1, so
    the errors are the probabilities' f16 roundings (2^-12 of themselves, or 2^-32 of the largest), the output's bf16 one,
    and fp32's: a score of 22 is off by 2^-19, the sum by 2^-13, 2^-12 together.  With token shares (one head) and without."""
    c = Paged(-(-n // 64), 64, 128, 16, 1, -(-n // 64))
    x = torch.zeros(n, c.row)
    x[0, 128] = 4.0
    x[1:, 0] = 1.0
    rows = [x.double()]
    for b in range(-(-n // 64)):
        part = x[b * 64:(b + 1) * 64].to(torch.bfloat16)
        c.pages[0, b, :len(part)] = part.to(DEV)
    c.table[0] = torch.arange(c.table.shape[1], dtype=torch.int32)
    c.lens[0] = n
    q = torch.zeros(1, heads, 80, dtype=torch.bfloat16, device=DEV)
    q[:, :, 64] = 4.0
    w = torch.zeros(heads, 128, 128, dtype=torch.bfloat16, device=DEV)
    w[:, 64:, 0] = 1.0
    scale = bits * math.log(2.0) / 16.0
    out = run_prefill(c, q, [0], [0, 1], heads, 64, 64, w, scale, n)
    assert c.bits() == 0
    ref, _, _ = attend64(q[0, :1].cpu().double(), torch.cat([torch.zeros(n, 64).double(), rows[0][:, 128:]], 1),
                         rows[0][:, :1].expand(n, 64), scale, [n])
    err = (out[0].cpu().double() - ref).abs()
    bound = (U + 2.0 ** -12 + 2.0 ** -12) * ref + n * 2.0 ** -32
    assert bool((err <= bound).all()), (float(err.max()), float(ref.max()), float(bound.max()))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("Q", [1, 3])
def test_a_query_that_sees_a_bad_latent_entry_is_nan_there(Q, bad):
    """Whatever the score becomes (with one infinite factor it is +infinity in some heads and -infinity in others), and
    whether or not every row of the tile sees the token: the entry is NaN, for a NaN all entries are."""
    heads = 6
    c = Paged(12, 32, 256, 32, 2, 6)
    c.fill([100, 129], seed=130)
    for s, t in ((0, 99), (1, 128)):
        c.pages[0, int(c.table[s, t // 32]), t % 32, 7] = bad
    q = make_q(2 * Q, heads, c.row, 131)
    q[:, ::2, 7] = q[:, ::2, 7].abs() + 0.1
    q[:, 1::2, 7] = -q[:, 1::2, 7].abs() - 0.1
    for scale in (0.1, -0.1):
        out, _ = run_decode(c, q, [0, 1], Q, heads, scale)
        assert c.bits() == 0
        seen = torch.arange(2 * Q, device=DEV) % Q == Q - 1
        assert bool(torch.isnan(out[seen][:, :, 7]).all()) and bool(torch.isfinite(out[~seen]).all())
        if bad != bad:
            assert bool(torch.isnan(out[seen]).all())


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_prefill_a_query_that_sees_a_bad_latent_entry_is_nan(sign):
    """An infinite latent makes all keys of its token infinite, and with keys of one sign and queries of one sign the score
    is +infinity or -infinity, not NaN by itself."""
    c = Paged(12, 32, 256, 32, 2, 6)
    q, w = make_q(60, 2, 96, 132), make_w(2, 128, 256, 133)
    q[:, :, :64] = sign * (q[:, :, :64].abs() + 0.1)
    w[:, :64, 7] = w[:, :64, 7].abs() + 0.1
    for bad in (float("inf"), float("-inf"), float("nan")):
        c.fill([100, 129], seed=134)
        for s, t in ((0, 99), (1, 120)):
            c.pages[0, int(c.table[s, t // 32]), t % 32, 7] = bad
        out = run_prefill(c, q, [0, 1], [0, 30, 60], 2, 64, 64, w, 0.1, 229)
        c.bits()                                   # an infinite value is beyond the f16 range: reported
        seen = torch.tensor([i == 29 or i >= 51 for i in range(60)], device=DEV)
        assert bool(torch.isnan(out[seen]).all()) and bool(torch.isfinite(out[~seen]).all())


def test_an_infinite_rotary_entry_leaves_its_token_out_or_is_nan():
    c = Paged(12, 32, 256, 32, 1, 6)
    rows = c.fill([90], seed=140)
    c.pages[0, int(c.table[0, 0]), 5, 256] = float("inf")
    q, qp, w = make_q(2, 4, c.row, 141), make_q(2, 2, 96, 142), make_w(2, 128, 256, 143)
    clean = {0: torch.cat([rows[0][:5], rows[0][6:]])}
    for sign in (1.0, -1.0):
        q[:, :, 256] = sign
        qp[:, :, 64] = sign
        out, _ = run_decode(c, q, [0], 2, 4, 0.1)
        outp = run_prefill(c, qp, [0], [0, 2], 2, 64, 64, w, 0.1, 90)
        assert c.bits() == 0
        if sign > 0:
            assert bool(torch.isnan(out).all()) and bool(torch.isnan(outp).all())
        else:
            check_decode(c, clean, q, [0], 2, 4, 0.1, out, None)
            check_prefill(c, clean, qp, [0], [0, 2], 2, 64, w, 0.1, outp)
