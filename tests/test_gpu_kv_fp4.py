"""The latent cache in 4 bits on the GPU: stored bytes and values bit for bit
against the look-up form in 64 bits, the page calls over its pages, and both
attention forms against 64 bits and, bit for bit, against a bf16 cache of the
values it stands for (the products take the same operands in the same order)."""
import math
import random

import numpy as np
import pytest
import torch

import edge_moe_serving_gb300 as moe
from fp4_helpers import Paged4, pack, unpack
from kv_helpers import DEV
from test_gpu_kv_pages import Pair, i32
from test_gpu_latent_attention import (DECODE, PREFILL, PREFIX, WIDTHS, check_decode, check_prefill, make_q, make_w,
                                       run_decode, run_prefill)

pytestmark = pytest.mark.gpu


def held(c, lens):
    """Sequences of those lengths on scattered pages, nothing stored yet."""
    c.fill([0] * len(lens))
    g = torch.Generator().manual_seed(5)
    order = torch.randperm(c.refs.numel(), generator=g).tolist()
    for i, n in enumerate(lens):
        for b in range(-(-n // c.page)):
            p = order.pop()
            c.table[i, b] = p
            c.refs[p] = 1
        c.lens[i] = n


def stored(c, layer=0):
    """The bytes of every token of every sequence, [sequence][token]."""
    out = []
    for s in range(c.lens.numel()):
        n = int(c.lens[s])
        ids = c.table[s, :-(-n // c.page)].long()
        out.append(c.pages[layer, ids].reshape(-1, c.bytes)[:n].cpu())
    return out


SHAPES = [
    # rank, rope, page, lens
    (512, 64, 16, [1]),
    (512, 64, 64, [65, 1, 700, 33]),
    (256, 32, 128, [129, 5]),
    (128, 64, 32, [40, 3, 77]),        # rows that end in zeros
    (384, 16, 16, [17, 50]),
    (32, 8, 16, [19]),
    (96, 0, 64, [70, 64]),
    (1024, 0, 32, [33]),               # more blocks than a warp has lanes
]


@pytest.mark.parametrize("rank,rope,page,lens", SHAPES)
def test_store_and_read(rank, rope, page, lens):
    c = Paged4(sum(-(-n // page) for n in lens) + 3, page, rank, rope, len(lens) + 1, -(-max(lens) // page), layers=2)
    held(c, lens)
    toks = [(s, t) for s, n in enumerate(lens) for t in range(n)]
    random.Random(rank).shuffle(toks)
    g = torch.Generator().manual_seed(rank + rope)
    rows = torch.randn(len(toks), rank + rope, generator=g) * torch.exp(2 * torch.randn(len(toks), 1, generator=g))
    rows = rows.to(torch.bfloat16)
    seq, pos = i32([s for s, _ in toks]), i32([t for _, t in toks])
    moe.moe_kv_append(c.handle, 1, rows.to(DEV), seq, pos, len(toks), c.status)
    want = pack(rows, rank, rope)
    got = stored(c, 1)
    for i, (s, t) in enumerate(toks):
        assert torch.equal(got[s][t], want[i]), (s, t)
    assert bool((c.pages[0] == 255).all())                       # the other layer
    back = torch.full((len(toks), rank + rope), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_read(c.handle, 1, seq, pos, len(toks), back, c.status)
    assert c.bits() == 0
    assert torch.equal(back.cpu().double(), unpack(want, rank, rope))


def special_rows(rank, rope):
    """Rows at the borders of the format: ties of codes and scales, zeros, subnormals, blocks beyond the largest scale."""
    rows = []
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0]
    for k in (8, 9, 11, 15):
        for e in (-17, -14, -11, -3, 0, 5, 11):
            rows.append([v * k * 2.0 ** e for v in ties])
    for k in (17, 19, 21, 31):                       # largest / 6 halfway between two scales
        for e in (-20, -19, -18, -5, 3):
            rows.append([6.0 * k * 2.0 ** e, 1.0 * k * 2.0 ** e, -2.0 ** e] + [0.0] * 13)
    rows += [[0.0] * 16, [-0.0] * 16, [2.0 ** -133] * 16, [2.0 ** -18 * 6, -2.0 ** -18] + [0.0] * 14,
             [2.0 ** -17 * 3, 2.0 ** -18] + [0.0] * 14, [2.0 ** -18 * 3, 1e-30] + [0.0] * 14, [368640.0] + [1.0] * 15]
    out = []
    for r in rows:
        out += r
    n = -(-len(out) // rank)
    out += [0.0] * (n * rank - len(out))
    x = torch.tensor(out, dtype=torch.float64).view(n, rank)
    return torch.cat([x, torch.arange(n * rope, dtype=torch.float64).view(n, rope)], 1).to(torch.bfloat16)


def test_store_at_the_borders():
    c = Paged4(4, 64, 512, 64, 1, 4)
    rows = special_rows(512, 64)
    n = len(rows)
    held(c, [n])
    seq, pos = i32([0] * n), i32(list(range(n)))
    moe.moe_kv_append(c.handle, 0, rows.to(DEV), seq, pos, n, c.status)
    assert c.bits() == 0
    want = pack(rows, 512, 64)
    got = stored(c)[0]
    assert torch.equal(unpack(got, 512, 64), unpack(want, 512, 64))
    assert torch.equal(got[:, 320:], want[:, 320:])              # the scales' bytes
    back = torch.empty(n, 576, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_read(c.handle, 0, seq, pos, n, back, c.status)
    assert torch.equal(back.cpu().double(), unpack(want, 512, 64))


def test_every_code_and_scale_is_read_as_it_stands():
    """All 256 scales, each with the 16 codes."""
    c = Paged4(16, 16, 512, 64, 1, 16)
    held(c, [8])
    data = torch.zeros(8, c.bytes, dtype=torch.uint8)
    codes = torch.tensor([2 * i + 16 * (2 * i + 1) for i in range(8)], dtype=torch.uint8)
    for r in range(8):
        data[r, :256] = codes.repeat(32)
        data[r, 384:416] = torch.arange(32 * r, 32 * r + 32, dtype=torch.uint8)
    c.pages[0, int(c.table[0, 0]), :8] = data.to(DEV)
    back = torch.empty(8, 576, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_read(c.handle, 0, i32([0] * 8), i32(list(range(8))), 8, back, c.status)
    want = unpack(data, 512, 64)
    got = back.cpu().double()
    nan = torch.isnan(want)
    assert bool((torch.isnan(got) == nan).all()) and bool(nan.any()) and torch.equal(got[~nan], want[~nan])


def test_store_beyond_the_range():
    c = Paged4(4, 16, 128, 16, 1, 2)
    held(c, [3])
    rows = torch.zeros(3, 144, dtype=torch.bfloat16)
    rows[0, 0], rows[0, 1], rows[0, 16] = 1e6, -3e38, 5.0        # clamped
    rows[1, 5], rows[1, 20] = float("nan"), 1.0
    rows[2, 40], rows[2, 41] = float("-inf"), 2.0
    moe.moe_kv_append(c.handle, 0, rows.to(DEV), i32([0] * 3), i32([0, 1, 2]), 3, c.status)
    assert c.bits() == moe.MOE_DEV_ERR_RANGE
    back = torch.empty(3, 144, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_read(c.handle, 0, i32([0] * 3), i32([0, 1, 2]), 3, back, c.status)
    assert c.bits() == 0
    back = back.cpu().double()
    assert back[0, 0] == 368640 and back[0, 1] == -368640 and abs(float(back[0, 16]) - 5.0) < 0.5
    assert bool(torch.isnan(back[1, :16]).all()) and bool(torch.isfinite(back[1, 16:]).all())
    assert bool(torch.isnan(back[2, 32:48]).all()) and bool(torch.isfinite(back[2, :32]).all())
    moe.moe_kv_append(c.handle, 0, rows[1:].to(DEV), i32([0] * 2), i32([1, 2]), 2, c.status)
    assert c.bits() == 0                                         # NaN and infinity alone are not out of range


@pytest.mark.parametrize("four", [True, False])
def test_refused_entries(four):
    from kv_helpers import Paged
    c = (Paged4 if four else Paged)(8, 16, 128, 16, 3, 3)
    rows0 = c.fill([20, 30], seed=4, shared_blocks=1)
    before = c.pages.clone()
    seq = i32([0, -1, 3, 0, 0, 1, 1, 2, 1])
    pos = i32([17, 0, 0, 20, -1, 0, 29, 0, 30])
    rows = torch.ones(9, 144, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_append(c.handle, 0, rows, seq, pos, 9, c.status)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ | moe.MOE_DEV_ERR_BAD_PAGE     # (1, 0) lies on a shared page
    same = before.view(torch.uint8) == c.pages.view(torch.uint8)
    same = same.view(*same.shape[:3], -1)
    changed = set(map(tuple, (~same.all(-1)).nonzero().tolist()))
    assert changed == {(0, int(c.table[0, 1]), 1), (0, int(c.table[1, 1]), 13)}
    back = torch.full((9, 144), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_read(c.handle, 0, seq, pos, 9, back, c.status)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    for i in (1, 2, 3, 4, 7, 8):
        assert bool((back[i] == 7).all())
    one = unpack(pack(rows[:1].cpu(), 128, 16), 128, 16)[0] if four else rows[0].cpu().double()
    assert torch.equal(back[0].cpu().double(), one) and torch.equal(back[6].cpu().double(), one)
    assert torch.equal(back[5].cpu().double(), rows0[1][0])      # shared pages can be read
    c.table[1, 1] = -1
    moe.moe_kv_read(c.handle, 0, i32([1, 0]), i32([29, 0]), 2, back, c.status)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_PAGE and torch.equal(back[1].cpu().double(), rows0[0][0])


def test_read_of_a_bf16_cache():
    from kv_helpers import Paged
    c = Paged(40, 16, 256, 32, 4, 16)
    rows = c.fill([100, 1, 33], seed=9)
    toks = [(s, t) for s in range(3) for t in range(len(rows[s]))]
    random.Random(1).shuffle(toks)
    back = torch.empty(len(toks), 288, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_read(c.handle, 0, i32([s for s, _ in toks]), i32([t for _, t in toks]), len(toks), back, c.status)
    assert c.bits() == 0
    assert torch.equal(back.cpu().double(), torch.stack([rows[s][t] for s, t in toks]))


class Pair4(Pair):
    """The page calls' model over a cache in 4 bits: a row is told by its rotary key, which is kept as it is."""

    def __init__(self, n_pages, page, max_seqs, max_blocks, layers):
        super().__init__(n_pages, page, max_seqs, max_blocks, layers, 32, 8)
        self.c = Paged4(n_pages, page, 32, 8, max_seqs, max_blocks, layers)

    def append(self, seqs, pos):
        n = len(seqs)
        ids = list(range(self.next_row, self.next_row + n))
        self.next_row += n
        for layer in range(self.c.pages.shape[0]):
            rows = torch.zeros(n, 40, dtype=torch.bfloat16, device=DEV)
            rows[:, :32] = i32(ids).view(-1, 1) % 7 - 3
            rows[:, 32:] = i32([i * 8 + layer for i in ids]).view(-1, 1).repeat(1, 4).view(torch.bfloat16)
            moe.moe_kv_append(self.c.handle, layer, rows, i32(seqs), i32(pos), n, self.c.status)
        for s, t, r in zip(seqs, pos, ids):
            self.m.append(s, t, r)

    def check(self, contents=True):
        super().check(False)
        data = self.c.pages.cpu()
        key = data[..., 16:32].contiguous().view(torch.int32)
        for s in range(len(self.m.lens)):
            for t, r in enumerate(self.m.rows(s)):
                if r is None:
                    continue
                at = self.m.table[s][t // self.c.page], t % self.c.page
                for layer in range(len(data)):
                    assert bool((key[layer][at] == r * 8 + layer).all()), (s, t)
                    got = unpack(data[layer][at][None], 32, 8)[0, :32]
                    want = unpack(pack(torch.full((1, 40), float(r % 7 - 3), dtype=torch.bfloat16), 32, 8), 32, 8)[0, :32]
                    assert torch.equal(got, want)


@pytest.mark.parametrize("page,layers,seed", [(16, 1, 0), (64, 3, 1)])
def test_page_calls(page, layers, seed):
    rng = random.Random(seed)
    p = Pair4(n_pages=60, page=page, max_seqs=9, max_blocks=7, layers=layers)
    for _ in range(40):
        op = rng.random()
        some = rng.sample(range(9), rng.randint(1, 5))
        if op < 0.45:
            before = list(p.m.lens)
            if p.reserve(some, [rng.choice([0, 1, page, rng.randint(0, 2 * page)]) for _ in some]):
                assert p.c.bits() == 0
                toks = [(s, t) for s in some for t in range(before[s], p.m.lens[s])]
                if toks:
                    p.append([s for s, _ in toks], [t for _, t in toks])
            else:
                assert p.c.bits() == moe.MOE_DEV_ERR_CAPACITY
        elif op < 0.7:
            ok = p.fork([rng.randrange(9) for _ in some], some)
            assert p.c.bits() == (0 if ok else moe.MOE_DEV_ERR_CAPACITY)
        elif op < 0.85:
            p.free(some)
        else:
            p.compact()
        p.check()


def test_page_calls_in_their_two_launch_forms():
    """Copies past 384 KB and pools past 8 MB."""
    p = Pair4(n_pages=4000, page=128, max_seqs=80, max_blocks=20, layers=2)
    p.reserve(list(range(40)), [100 + 13 * i for i in range(40)])
    toks = [(s, t) for s in range(0, 40, 7) for t in range(p.m.lens[s])]
    p.append([s for s, _ in toks], [t for _, t in toks])
    p.fork(list(range(40)), list(range(40, 80)))
    p.free(list(range(0, 40, 3)))
    p.compact()
    p.check()
    assert p.c.bits() == 0


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("rank,rope,page,heads,Q,lens", DECODE)
def test_decode(rank, rope, page, heads, Q, lens):
    blocks = [-(-n // page) for n in lens]
    c = Paged4(sum(blocks) + 5, page, rank, rope, len(lens) + 2, max(blocks) + 1)
    rows = c.fill(lens, seed=heads)
    q = make_q(len(lens) * Q, heads, c.row, 3)
    scale = 1.0 / math.sqrt(128 + rope)
    seqs = list(range(len(lens)))[::-1]
    out, lse = run_decode(c, q, seqs, Q, heads, scale)
    assert c.bits() == 0
    check_decode(c, rows, q, seqs, Q, heads, scale, out, lse)
    twin, twin_lse = run_decode(c.twin(), q, seqs, Q, heads, scale)
    assert torch.equal(out, twin) and torch.equal(lse, twin_lse)
    again, _ = run_decode(c, q, seqs, Q, heads, scale, lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("rank,rope,page,heads,Q,shared_blocks,own", PREFIX)
def test_shared_prefix(rank, rope, page, heads, Q, shared_blocks, own):
    shared = shared_blocks * page
    lens = [shared + n for n in own]
    blocks = [-(-n // page) for n in lens]
    c = Paged4(sum(blocks) + 5, page, rank, rope, len(lens), max(blocks))
    rows = c.fill(lens, seed=heads, shared_blocks=shared_blocks)
    q = make_q(len(lens) * Q, heads, c.row, 4)
    scale = 1.0 / math.sqrt(128 + rope)
    seqs = list(range(len(lens)))
    out, lse = run_decode(c, q, seqs, Q, heads, scale, shared=shared)
    assert c.bits() == 0
    check_decode(c, rows, q, seqs, Q, heads, scale, out, lse)
    twin, twin_lse = run_decode(c.twin(), q, seqs, Q, heads, scale, shared=shared)
    assert torch.equal(out, twin) and torch.equal(lse, twin_lse)


@pytest.mark.parametrize("B,heads,first", [(40, 64, 0), (600, 8, 0), (40, 64, -1)])
def test_a_prefix_of_many_row_tiles(B, heads, first):
    """Enough row tiles over the shared tokens that these are expanded once for all of them (at 600 sequences in the first
    of two launches alone); sequences that end inside the shared tokens and behind them; a bad first id."""
    shared, page = 6400, 64
    c = Paged4(110, page, 128, 16, B, 104, layers=2)
    rows = c.fill([shared + 100], seed=B, layer=1)[0]
    c.table[1:] = c.table[:1]
    lens = [shared + 100 - (i * 7) % 150 for i in range(B)]
    c.lens.copy_(i32(lens))
    q = make_q(B, heads, c.row, 4)
    seqs = list(range(B))
    seqs[0] = first
    out, lse = run_decode(c, q, seqs, 1, heads, 0.1, shared=shared, layer=1)
    if first < 0:
        assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ and bool((out == 0).all()) and bool((lse == -math.inf).all())
        return
    assert c.bits() == 0
    twin, twin_lse = run_decode(c.twin(), q, seqs, 1, heads, 0.1, shared=shared, layer=1)
    assert torch.equal(out, twin) and torch.equal(lse, twin_lse)
    for b in (0, 1, 17, B - 1):
        check_decode(c, {b: rows[:lens[b]]}, q[b:b + 1], [b], 1, heads, 0.1, out[b:b + 1], lse[b:b + 1])
    c.table[:, 3] = 10 ** 6
    run_decode(c, q, seqs, 1, heads, 0.1, shared=shared, layer=1)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_PAGE


def test_decode_of_many_sequences_and_layers():
    """More sequences than one launch takes, empty ones among them, in the second of three layers."""
    lens = [(i * 37) % 150 for i in range(600)]
    c = Paged4(2 + sum(-(-n // 32) for n in lens), 32, 128, 16, 600, 5, layers=3)
    rows = c.fill(lens, seed=60, layer=1)
    q = make_q(600, 5, c.row, 61)
    out, lse = run_decode(c, q, list(range(600)), 1, 5, 0.1, layer=1)
    assert c.bits() == 0
    some = [0, 1, 2, 511, 512, 513, 599]
    for b in some:
        check_decode(c, rows, q[b:b + 1], [b], 1, 5, 0.1, out[b:b + 1], lse[b:b + 1])


@pytest.mark.parametrize("Q", [1, 3])
def test_a_nan_block_reaches_the_queries_that_see_it(Q):
    c = Paged4(12, 32, 256, 32, 2, 6)
    rows = c.fill([100, 129], seed=130)
    for s, t in ((0, 99), (1, 128)):
        c.pages[0, int(c.table[s, t // 32]), t % 32, 128 + 64 + 1] = 0xFF      # the second scale
    q = make_q(2 * Q, 6, c.row, 131)
    out, _ = run_decode(c, q, [0, 1], Q, 6, 0.1)
    assert c.bits() == 0
    for b, n in ((0, 100), (1, 129)):
        for i in range(Q):
            at = b * Q + i
            if i == Q - 1:
                assert bool(torch.isnan(out[at]).all())
            else:
                check_decode(c, {b: rows[b][:n - Q + i + 1]}, q[at:at + 1], [b], 1, 6, 0.1, out[at:at + 1], None)


def test_decode_refused_on_the_device():
    c = Paged4(20, 64, 512, 64, 4, 6)
    rows = c.fill([100, 200, 30], seed=40)
    q = make_q(3, 16, c.row, 41)
    out, lse = run_decode(c, q, [0, 7, 2], 1, 16, 0.07)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    check_decode(c, rows, q[:1], [0], 1, 16, 0.07, out[:1], lse[:1])
    check_decode(c, rows, q[2:], [2], 1, 16, 0.07, out[2:], lse[2:])
    c.table[1, 2] = 77
    out, lse = run_decode(c, q, [0, 1, 2], 1, 16, 0.07)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_PAGE
    check_decode(c, rows, q[2:], [2], 1, 16, 0.07, out[2:], lse[2:])


@pytest.mark.parametrize("rank,rope,page,heads,dn,dv,lens,new", PREFILL + WIDTHS)
def test_prefill(rank, rope, page, heads, dn, dv, lens, new):
    blocks = [-(-n // page) for n in lens]
    c = Paged4(sum(blocks) + 5, page, rank, rope, len(lens) + 1, max(blocks) + 1)
    rows = c.fill(lens, seed=heads)
    seqs = list(range(len(lens)))
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    q, w = make_q(offsets[-1], heads, dn + rope, 12), make_w(heads, dn + dv, rank, 13)
    scale = 1.0 / math.sqrt(dn + rope)
    out = run_prefill(c, q, seqs, offsets, heads, dn, dv, w, scale, sum(lens))
    assert c.bits() == 0
    check_prefill(c, rows, q, seqs, offsets, heads, dn, w, scale, out)
    assert torch.equal(out, run_prefill(c.twin(), q, seqs, offsets, heads, dn, dv, w, scale, sum(lens)))


def test_prefill_refused_on_the_device():
    c = Paged4(20, 64, 512, 64, 4, 6)
    rows = c.fill([100, 200, 30], seed=40)
    q, w = make_q(60, 2, 192, 41), make_w(2, 256, 512, 42)
    out = run_prefill(c, q, [0, 1], [0, 20, 60], 2, 128, 128, w, 0.07, 20)
    assert c.bits() == moe.MOE_DEV_ERR_CAPACITY and bool(torch.isnan(out).all())
    c.table[1, 3] = -1
    out = run_prefill(c, q, [0, 1], [0, 20, 60], 2, 128, 128, w, 0.07, 300)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_PAGE
    check_prefill(c, rows, q[:20], [0], [0, 20], 2, 128, w, 0.07, out[:20])


def test_store_and_attend_in_a_graph_on_another_stream():
    """A decode step (a row stored, then attended to) captured once and replayed as the sequences grow."""
    c = Paged4(40, 16, 512, 64, 2, 12)
    rows = c.fill([60, 110], seed=70)
    q = make_q(2, 16, c.row, 71)
    new = make_q(3, 2, c.row, 72)
    seqs, pos, row = i32([0, 1]), i32([60, 110]), new[0].clone()
    n = moe.moe_latent_decode_workspace_size(c.handle, 2, 1, 16, 0)
    ws, out = torch.zeros(n, dtype=torch.uint8, device=DEV), torch.zeros(2, 16, 512, dtype=torch.bfloat16, device=DEV)
    one = i32([1, 1])
    s = torch.cuda.Stream()

    def step():
        moe.moe_kv_reserve(c.handle, seqs, one, 2, c.ws, c.ws.numel(), c.status)
        moe.moe_kv_append(c.handle, 0, row, seqs, pos, 2, c.status)
        moe.moe_latent_decode(c.handle, 0, q, seqs, 2, 1, 16, 0.07, 0, out, None, ws, n, c.status)

    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        step()
    for i in range(3):
        row.copy_(new[i])
        g.replay()
        pos += 1
        torch.cuda.synchronize()
        for b in range(2):
            rows[b] = torch.cat([rows[b], unpack(pack(new[i, b:b + 1].cpu(), 512, 64), 512, 64)])
        check_decode(c, rows, q, [0, 1], 1, 16, 0.07, out, None)
    assert c.bits() == 0 and np.array_equal(c.lens.cpu().numpy()[:2], [63, 113])
