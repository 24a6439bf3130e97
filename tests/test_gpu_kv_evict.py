"""Eviction by attention weight: tables, lengths, reference counts, rows, weights
and kept positions bit-exact against a model on lists."""
import random

import numpy as np
import pytest
import torch

import edge_moe_serving_gb300 as moe
from fp4_helpers import Paged4
from kv_helpers import DEV, Paged
from test_gpu_latent_attention import check_decode, make_q, run_decode
from test_gpu_latent_weights import run_weights

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def heaviest_first(w, t):
    return (0, 0.0, t) if np.isnan(w) else (1, -float(w), t)


def model(c, state, seqs, budget, first, recent):
    """What the header says, on copies: {name: array}; kept[layer, i] lists the positions."""
    pages, table, lens, refs, weights = (x.copy() for x in state)
    before, refs0 = pages.copy(), refs.copy()
    layers, cap = pages.shape[0], weights.shape[2]
    kept = np.full((layers, len(seqs), cap), -7, np.int32)
    seen = set()
    for i, s in enumerate(seqs):
        if not 0 <= s < len(lens) or s in seen:
            continue
        seen.add(s)
        n = int(lens[s])
        ids = table[s, :-(-n // c.page)].copy()
        head = tail = n
        if n > budget:
            if (ids < 0).any() or (ids >= len(refs)).any():
                continue
            shared = [b + 1 for b, p in enumerate(ids) if refs0[p] > 1]
            head = min(n, max(first, max(shared, default=0) * c.page))
            tail = max(head, n - recent)
        now = max(budget, head + n - tail) if n > budget else n
        for layer in range(layers):
            w = weights[layer, s]
            middle = sorted(range(head, tail), key=lambda t: heaviest_first(w[t], t))[:now - head - (n - tail)]
            keep = list(range(head)) + sorted(middle) + list(range(tail, n))
            if n <= budget:
                keep = list(range(n))
            kept[layer, i, :now] = keep
            for j, t in enumerate(keep):
                pages[layer, ids[j // c.page], j % c.page] = before[layer, ids[t // c.page], t % c.page]
            w[:n] = np.concatenate([w[keep], np.zeros(n - now, np.float32)])
        for b in range(-(-now // c.page), len(ids)):
            refs[ids[b]] -= 1
            table[s, b] = -1
        lens[s] = now
    return pages, table, lens, refs, weights, kept


def state_of(c, weights):
    pages = c.pages.view(torch.uint8) if c.pages.dtype != torch.uint8 else c.pages
    return [x.cpu().numpy().copy() for x in (pages, c.table, c.lens, c.refs, weights)]


def run(c, seqs, weights, budget, first, recent, kept=True, stream=None):
    layers = c.pages.shape[0]
    k = torch.full((layers, len(seqs), weights.shape[2]), -7, dtype=torch.int32, device=DEV) if kept else None
    n = moe.moe_kv_evict_workspace_size(c.handle, len(seqs))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    moe.moe_kv_evict(c.handle, i32(seqs), len(seqs), weights, budget, first, recent, k, ws, n, c.status, stream)
    return k


def make(lens, page, layers=1, rank=64, rope=8, seed=0, shared_blocks=0, four=False, spare=3, max_blocks=None):
    blocks = [-(-n // page) for n in lens]
    c = (Paged4 if four else Paged)(sum(blocks) + spare, page, rank, rope, len(lens) + 1, max_blocks or max(blocks) + 1, layers)
    c.fill(lens, seed=seed, shared_blocks=shared_blocks)
    g = torch.Generator(device=DEV).manual_seed(seed)
    c.pages.view(torch.uint8).random_(0, 256, generator=g)       # every row is its own, in every layer
    w = torch.randn(layers, len(lens) + 1, c.table.shape[1] * page, generator=g, device=DEV).mul(2).exp()
    return c, w


def check(c, w, seqs, budget, first, recent, bits=0, kept=True):
    before = state_of(c, w)
    want = model(c, before, seqs, budget, first, recent)
    k = run(c, seqs, w, budget, first, recent, kept)
    assert c.bits() == bits
    got = state_of(c, w) + ([k.cpu().numpy()] if kept else [])
    for name, a, b in zip(("pages", "table", "lens", "refs", "weights", "kept"), got, want):
        same = a.view(np.uint8) == b.view(np.uint8) if a.dtype == np.float32 else a == b
        assert same.all(), (name, np.argwhere(~same)[:5])


CASES = [
    # lens, page, layers, budget, first, recent, shared blocks
    ([5], 16, 1, 3, 0, 0, 0),
    ([2], 16, 1, 1, 1, 0, 0),
    ([100, 33, 20, 0, 64], 16, 2, 32, 2, 8, 0),
    ([100, 33, 20, 17], 16, 3, 17, 0, 17, 0),                # the newest tokens alone
    ([300, 299, 301, 256], 32, 1, 256, 4, 64, 0),
    ([300, 200, 500], 32, 2, 100, 0, 0, 0),
    ([700, 650, 620, 640], 64, 2, 600, 4, 32, 5),
    ([700, 650, 620, 640], 64, 1, 300, 4, 32, 8),            # shared tokens beyond the budget: all of them stay
    ([512, 512, 512], 128, 1, 512, 0, 0, 3),                 # nothing to do
    ([640, 640, 640], 128, 2, 512, 0, 0, 5),                 # every token is shared
    ([5000, 4100, 2049, 1025], 64, 1, 1024, 1, 100, 0),
    ([9000], 128, 2, 8999, 4, 10, 0),                        # a single token goes
    ([40000, 33000], 128, 1, 20000, 4, 1000, 2),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("lens,page,layers,budget,first,recent,shared", CASES)
def test_evict(lens, page, layers, budget, first, recent, shared, four):
    c, w = make(lens, page, layers, seed=len(lens), shared_blocks=shared, four=four)
    check(c, w, list(range(len(lens)))[::-1], budget, first, recent)


@pytest.mark.parametrize("rank,rope,four", [(512, 64, False), (512, 64, True), (128, 16, True), (384, 16, True), (8, 0, False),
                                            (2048, 64, False)])
def test_row_widths(rank, rope, four):
    c, w = make([500, 130, 77], 16, 2, rank, rope, seed=rank, four=four)
    check(c, w, [0, 2, 1], 96, 3, 20, kept=False)


def test_ties_and_unusual_weights():
    """Equal weights, zeros of both signs, negative ones, infinities and NaN."""
    for seed in range(4):
        c, w = make([400, 333, 250], 16, 2, seed=seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        values = torch.tensor([0.0, -0.0, 1.0, 1.0, -1.0, 2.0, float("inf"), float("nan"), -float("inf"), 1e-40], device=DEV)
        w.copy_(values[torch.randint(0, [3, 5, 10, 10][seed], w.shape, generator=g, device=DEV)])
        check(c, w, [1, 0, 2], [100, 200, 37, 240][seed], 2, 16)
    c, w = make([400, 333], 16, 1)
    w.zero_()
    check(c, w, [0, 1], 64, 0, 0)                            # all alike: the first ones stay


def test_layers_choose_for_themselves():
    c, w = make([200], 16, 4, seed=3)
    k = run(c, [0], w, 50, 1, 5)
    assert c.bits() == 0 and len({tuple(x) for x in k[:, 0, :50].tolist()}) == 4


def test_refused_entries():
    c, w = make([200, 150, 170], 16, 2, seed=5)
    check(c, w, [1, 7, 1, 0], 64, 2, 8, bits=moe.MOE_DEV_ERR_BAD_SEQ)
    check(c, w, [-1, 2, 2, 4], 50, 2, 8, bits=moe.MOE_DEV_ERR_BAD_SEQ)
    c, w = make([200, 150, 170], 16, 2, seed=6)
    c.table[1, 4] = -1
    check(c, w, [0, 1, 2], 64, 2, 8, bits=moe.MOE_DEV_ERR_BAD_PAGE)
    c, w = make([200, 150, 170], 16, 2, seed=7)
    c.table[0, 3] = 10 ** 6
    check(c, w, [0, 1, 2], 64, 2, 8, bits=moe.MOE_DEV_ERR_BAD_PAGE)


def test_lengths_past_the_blocks_are_cut():
    """A length that the block table has no room for counts up to its end."""
    c, w = make([128], 16, 1, max_blocks=8)
    c.lens[0] = 5000
    before = state_of(c, w)
    before[2][0] = 128
    want = model(c, before, [0], 50, 1, 5)
    run(c, [0], w, 50, 1, 5)
    assert c.bits() == 0
    for a, b in zip(state_of(c, w), want):
        assert (a.view(np.uint8) == b.view(np.uint8)).all()


@pytest.mark.parametrize("seed", range(6))
def test_random(seed):
    rng = random.Random(seed)
    page = rng.choice([16, 32, 64, 128])
    shared = rng.choice([0, 0, 1, 3])
    lens = [shared * page + rng.randint(0, 900) for _ in range(rng.randint(1, 12))]
    budget = rng.randint(1, 700)
    first = rng.randint(0, min(budget, 9))
    c, w = make(lens, page, rng.choice([1, 2, 3]), rng.choice([64, 256, 512]), 64, seed=seed, shared_blocks=shared,
                four=rng.random() < 0.5)
    seqs = rng.sample(range(len(lens)), rng.randint(1, len(lens)))
    check(c, w, seqs, budget, first, rng.randint(0, budget - first))


@pytest.mark.parametrize("four", [False, True])
def test_a_serving_step(four):
    """Decode, weights, eviction, a new token, decode again: the second answer is attention over the tokens that stayed."""
    c = (Paged4 if four else Paged)(80, 32, 256, 32, 3, 24)
    lens = [600, 250, 410]
    rows = c.fill(lens, seed=21)
    q, scale, heads = make_q(3, 12, c.row, 22), 0.1, 12
    w = torch.zeros(1, 3, 24 * 32, device=DEV)
    _, lse = run_decode(c, q, [0, 1, 2], 1, heads, scale)
    run_weights(c, q, [0, 1, 2], 1, heads, scale, lse, 1.0, w[0])
    k = run(c, [0, 1, 2], w, 256, 4, 32)
    assert c.lens.tolist() == [256, 250, 256]
    rows = [x[k[0, s, :n].cpu().long()] for s, (x, n) in enumerate(zip(rows, c.lens.tolist()))]
    moe.moe_kv_reserve(c.handle, i32([0, 1, 2]), i32([1, 1, 1]), 3, c.ws, c.ws.numel(), c.status)
    new = make_q(3, 1, c.row, 23).view(3, -1)
    moe.moe_kv_append(c.handle, 0, new, i32([0, 1, 2]), i32([256, 250, 256]), 3, c.status)
    back = torch.empty_like(new)
    moe.moe_kv_read(c.handle, 0, i32([0, 1, 2]), i32([256, 250, 256]), 3, back, c.status)
    rows = [torch.cat([x, back[s:s + 1].cpu().double()]) for s, x in enumerate(rows)]
    assert bool((w[0, [0, 1, 2], [256, 250, 256]] == 0).all())       # a new token starts without weight
    q = make_q(3, heads, c.row, 24)
    out, lse = run_decode(c, q, [0, 1, 2], 1, heads, scale)
    assert c.bits() == 0
    check_decode(c, rows, q, [0, 1, 2], 1, heads, scale, out, lse)


def test_in_a_graph_on_another_stream():
    c, w = make([300, 200], 16, 2, seed=8)
    first = state_of(c, w)
    n = moe.moe_kv_evict_workspace_size(c.handle, 2)
    ws, seqs = torch.zeros(n, dtype=torch.uint8, device=DEV), i32([0, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_kv_evict(c.handle, seqs, 2, w, 128, 2, 16, None, ws, n, c.status)
    pages = c.pages.view(torch.uint8)
    for lens in ([300, 200], [150, 100]):
        for t, x in zip((pages, c.table, c.lens, c.refs, w), first):
            t.copy_(torch.from_numpy(x))
        c.lens[:2] = i32(lens)
        before = state_of(c, w)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(state_of(c, w), model(c, before, [0, 1], 128, 2, 16)):
            assert (a.view(np.uint8) == b.view(np.uint8)).all()
    assert c.bits() == 0
