"""The page calls of the latent cache against a plain model on lists: block
tables, lengths, reference counts and row contents bit-exact."""
import random

import numpy as np
import pytest
import torch

import edge_moe_serving_gb300 as moe
from kv_helpers import DEV, Model, Paged

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Pair:
    """The library's cache and the model, driven alike."""

    def __init__(self, n_pages, page, max_seqs, max_blocks, layers, rank=16, rope=8):
        self.c = Paged(n_pages, page, rank, rope, max_seqs, max_blocks, layers)
        self.m = Model(n_pages, page, max_seqs, max_blocks)
        self.next_row = 1

    def reserve(self, seqs, n_new):
        moe.moe_kv_reserve(self.c.handle, i32(seqs), i32(n_new), len(seqs), self.c.ws, self.c.ws.numel(), self.c.status)
        return self.m.reserve(seqs, n_new)

    def append(self, seqs, pos):
        n = len(seqs)
        ids = list(range(self.next_row, self.next_row + n))
        self.next_row += n
        layers = self.c.pages.shape[0]
        for layer in range(layers):
            rows = i32([i * 8 + layer for i in ids]).view(-1, 1).repeat(1, self.c.row // 2).view(torch.bfloat16)
            moe.moe_kv_append(self.c.handle, layer, rows.contiguous(), i32(seqs), i32(pos), n, self.c.status)
        for s, t, r in zip(seqs, pos, ids):
            self.m.append(s, t, r)

    def fork(self, src, dst):
        moe.moe_kv_fork(self.c.handle, i32(src), i32(dst), len(src), self.c.ws, self.c.ws.numel(), self.c.status)
        return self.m.fork(src, dst)

    def free(self, seqs):
        moe.moe_kv_free(self.c.handle, i32(seqs), len(seqs), self.c.status)
        self.m.free(seqs)

    def compact(self):
        n = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_kv_compact(self.c.handle, n, self.c.ws, self.c.ws.numel(), self.c.status)
        assert int(n.item()) == self.m.compact()

    def check(self, contents=True):
        m, c = self.m, self.c
        table = np.full(tuple(c.table.shape), -1, np.int32)
        for s, t in enumerate(m.table):
            table[s, :len(t)] = t
        assert np.array_equal(c.table.cpu().numpy(), table)
        assert c.lens.tolist() == m.lens
        assert c.refs.tolist() == m.refs
        if not contents:
            return
        words = c.pages.cpu().view(torch.int32)                        # [layers, pages, page, row / 2]
        for s in range(len(m.lens)):
            for t, r in enumerate(m.rows(s)):
                if r is not None:
                    got = words[:, m.table[s][t // c.page], t % c.page]
                    for layer in range(words.shape[0]):
                        assert bool((got[layer] == r * 8 + layer).all()), (s, t)


@pytest.mark.parametrize("page,layers,seed", [(16, 1, 0), (32, 3, 1), (64, 2, 2), (128, 1, 3)])
def test_random_trace(page, layers, seed):
    rng = random.Random(seed)
    p = Pair(n_pages=97, page=page, max_seqs=13, max_blocks=9, layers=layers)
    for _ in range(60):
        op = rng.random()
        some = rng.sample(range(13), rng.randint(1, 6))
        if op < 0.4:
            n_new = [rng.choice([0, 1, 2, page - 1, page, page + 1, rng.randint(0, 2 * page)]) for _ in some]
            before = list(p.m.lens)
            if p.reserve(some, n_new):
                assert p.c.bits() == 0
                toks = [(s, t) for s in some for t in range(before[s], p.m.lens[s])]
                if toks:
                    p.append([s for s, _ in toks], [t for _, t in toks])
            else:
                assert p.c.bits() == moe.MOE_DEV_ERR_CAPACITY
        elif op < 0.7:
            src = [rng.randrange(13) for _ in some]
            ok = p.fork(src, some)
            assert p.c.bits() == (0 if ok else moe.MOE_DEV_ERR_CAPACITY)
        elif op < 0.85:
            p.free(some)
            assert p.c.bits() == 0
        else:
            p.compact()
            assert p.c.bits() == 0
        p.check()


def test_beams_permute_and_fan_out():
    p = Pair(n_pages=64, page=16, max_seqs=4, max_blocks=8, layers=2)
    p.reserve([0, 1, 2, 3], [17, 33, 16, 40])
    for s, n in enumerate([17, 33, 16, 40]):
        p.append([s] * n, list(range(n)))
    p.check()
    p.fork([1, 0, 3, 2], [0, 1, 2, 3])       # swaps
    p.check()
    p.fork([2, 2, 2, 2], [0, 1, 2, 3])       # all follow one, which stays
    p.check()
    p.fork([3, 0, 1, 2], [0, 1, 2, 3])
    p.check()
    assert p.c.bits() == 0


def test_large_pool_and_lists():
    """More pages than one scan round, lists longer than a CTA, and a pool filled to its last page."""
    p = Pair(n_pages=9001, page=16, max_seqs=2100, max_blocks=5, layers=1, rank=8, rope=0)
    seqs = list(range(2100))
    assert p.reserve(seqs, [33 + (s % 3) * 16 for s in seqs])
    p.free(seqs[1::2])
    assert p.fork(seqs[0:2000:2], seqs[1:2000:2])
    p.check(contents=False)
    p.compact()
    p.check(contents=False)
    spare = p.m.refs.count(0)
    p.free([2001])
    spare = p.m.refs.count(0)
    empty = [s for s in seqs if p.m.lens[s] == 0]
    take = [16 * min(5, max(0, spare - 5 * i)) for i in range(len(empty))]
    ok = p.reserve(empty, take)
    p.check(contents=False)
    assert p.c.bits() == (0 if ok else moe.MOE_DEV_ERR_CAPACITY)


def test_refused_entries_and_full_pool():
    p = Pair(n_pages=6, page=16, max_seqs=5, max_blocks=3, layers=1)
    p.reserve([0, 7, -1, 1, 0], [20, 5, 5, 3, 9])                       # ids out of range, a repeat
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    p.check()
    p.reserve([2], [-1])
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    for seqs, n in (([2, 3], [48, 1]), ([2], [49])):                    # one page short; one block too many
        assert not p.reserve(seqs, n)
        assert p.c.bits() == moe.MOE_DEV_ERR_CAPACITY
        p.check()
    assert p.reserve([2], [48])
    p.check()
    assert not p.fork([0], [3])                                         # no page for the partial copy
    assert p.c.bits() == moe.MOE_DEV_ERR_CAPACITY
    p.check()
    assert p.fork([2, 9, 2], [3, 0, 3])                                 # whole pages only; a bad id; a repeat
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    p.check()
    p.free([3, 3, 8])
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    p.check()
    rows = torch.zeros(4, p.c.row, dtype=torch.bfloat16, device=DEV)
    before = p.c.pages.clone().view(torch.int16)
    moe.moe_kv_append(p.c.handle, 0, rows, i32([0, 9, 0, -1]), i32([20, 0, -1, 0]), 4, p.c.status)
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    p.fork([2], [3])
    moe.moe_kv_append(p.c.handle, 0, rows[:1], i32([2]), i32([3]), 1, p.c.status)   # a shared page
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_PAGE
    assert torch.equal(before, p.c.pages.view(torch.int16))


def test_nan_rows_are_copied_and_empty_lists_are_no_ops():
    p = Pair(n_pages=8, page=16, max_seqs=4, max_blocks=4, layers=1)
    n0 = moe.moe_kernel_launch_count()
    p.reserve([], [])
    p.fork([], [])
    p.free([])
    assert moe.moe_kernel_launch_count() == n0
    p.reserve([0], [5])
    rows = torch.full((5, p.c.row), float("nan"), dtype=torch.bfloat16, device=DEV)
    moe.moe_kv_append(p.c.handle, 0, rows, i32([0] * 5), i32(list(range(5))), 5, p.c.status)
    p.c.pages[0, 1] = 7.0                                               # where the copy goes
    p.fork([0], [1])
    got = p.c.pages[0, int(p.c.table[1, 0])]
    assert bool(torch.isnan(got[:5]).all()) and bool((got[5:] == 7.0).all())   # valid rows only
    p.fork([3], [1])                                                    # an empty source empties the destination
    p.check(contents=False)
    assert p.c.bits() == 0


def test_calls_in_a_graph_on_another_stream():
    p = Pair(n_pages=40, page=16, max_seqs=8, max_blocks=4, layers=1)
    p.reserve([0, 1], [20, 35])
    src, dst = i32([0, 1]), i32([4, 5])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_kv_fork(p.c.handle, src, dst, 2, p.c.ws, p.c.ws.numel(), p.c.status, s)
    p.m.fork([0, 1], [4, 5])
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_kv_fork(p.c.handle, src, dst, 2, p.c.ws, p.c.ws.numel(), p.c.status)
        moe.moe_kv_compact(p.c.handle, None, p.c.ws, p.c.ws.numel(), p.c.status)
    for _ in range(3):
        g.replay()
        p.m.fork([0, 1], [4, 5])
        p.m.compact()
    torch.cuda.synchronize()
    p.check(contents=False)
    assert p.c.bits() == 0


@pytest.mark.parametrize("n", [9728, 9729, 20001, 330007])
def test_append_of_many_rows(n):
    """Up to 9728 rows a warp of the grid takes one row at a time, beyond that up to 32, and beyond 311296 of them it
    comes back for more (152 SMs).  Tokens in any order, some entries that are refused among them."""
    seqs, page = 41, 128
    lens = [n // seqs + (i < n % seqs) for i in range(seqs)]
    blocks = [-(-k // page) for k in lens]
    c = Paged(sum(blocks), page, 16, 8, seqs, max(blocks), layers=2)
    moe.moe_kv_reserve(c.handle, i32(range(seqs)), i32(lens), seqs, c.ws, c.ws.numel(), c.status)
    order = np.random.RandomState(n).permutation(n)
    tok_seq = np.repeat(np.arange(seqs), lens)[order]
    tok_pos = np.concatenate([np.arange(k) for k in lens])[order]
    words = torch.from_numpy(np.random.RandomState(1).randint(0, 1 << 30, (n, c.row // 2)).astype(np.int32)).to(DEV)
    s, t = i32(tok_seq), i32(tok_pos)
    refused = torch.arange(7, n, 1009, device=DEV)
    s_in, t_in = s.clone(), t.clone()
    s_in[refused[::2]] = seqs
    t_in[refused[1::2]] = 1 << 20
    moe.moe_kv_append(c.handle, 1, words.view(torch.bfloat16), s_in, t_in, n, c.status)
    assert c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    got = c.pages.view(torch.int32)[1, c.table[s.long(), t.long() // page].long(), t.long() % page]
    want = words.clone()
    want[refused] = torch.full((c.row,), float("nan"), dtype=torch.bfloat16, device=DEV).view(torch.int32)
    assert torch.equal(got, want)
    assert bool(torch.isnan(c.pages[0]).all())


@pytest.mark.parametrize("seed", [5, 6])
def test_large_pools_and_copies(seed):
    """Forks and compactions whose bytes take the whole GPU (a plan and a second launch) instead of one cluster: a pool
    of 9.2 MB (above 8 MB), forks of 27 to 36 pairs of 15,360 bytes (above 384 KB), in place and onto empty sequences."""
    rng = random.Random(seed)
    p = Pair(n_pages=600, page=64, max_seqs=40, max_blocks=20, layers=5)
    assert 5 * 600 * 64 * p.c.row * 2 > 8 << 20 and 27 * 5 * 64 * p.c.row * 2 > 384 << 10
    for turn in range(4):
        empty = [s for s in range(40) if p.m.lens[s] == 0]
        new = rng.sample(empty, min(14, len(empty)))
        n_new = [rng.choice([1, 63, 64, 65, rng.randint(1, 900)]) for _ in new]
        assert p.reserve(new, n_new)
        toks = [(s, t) for s, n in zip(new, n_new) for t in range(n)]
        p.append([s for s, _ in toks], [t for _, t in toks])
        dst = rng.sample(range(40), rng.randint(27, 36))
        assert p.fork([rng.randrange(40) for _ in dst], dst)
        p.check(contents=turn == 1)
        p.free(rng.sample(range(40), 22))
        p.check(contents=False)
        p.compact()
        p.check(contents=turn == 3)
    assert p.c.bits() == 0


def test_a_large_fork_that_is_refused():
    """The two-launch form with too few free pages, bad ids and a source whose last page is missing."""
    p = Pair(n_pages=64, page=64, max_seqs=32, max_blocks=4, layers=5)
    p.reserve(list(range(30)), [65] * 30)
    assert not p.fork([0] * 27, list(range(1, 28)))                     # 27 partial pages, 4 free
    assert p.c.bits() == moe.MOE_DEV_ERR_CAPACITY
    p.check()
    p.free(list(range(3, 30)))
    src, dst = [0] * 27, list(range(3, 30))
    src[4], dst[9], dst[11] = 32, -1, 3                                 # a bad source, a bad destination, a repeat
    assert p.fork(src, dst)
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_SEQ
    p.check()
    p.c.table[0, 1] = -1
    moe.moe_kv_fork(p.c.handle, i32([0] * 28), i32([31] + [1] * 27), 28, p.c.ws, p.c.ws.numel(), p.c.status)
    assert p.c.bits() == moe.MOE_DEV_ERR_BAD_PAGE | moe.MOE_DEV_ERR_BAD_SEQ
