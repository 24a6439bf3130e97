"""Eviction in the form of large calls, whose CTAs move 128 bytes of every row
(those of small calls move 32): rows whose bytes are no multiple of 128, shared
pages in front, sequences longer than a CTA keeps the weights of in registers
(8192 tokens), repeats and refused ids.  Exact, against the model on lists."""
import pytest
import torch

import edge_moe_serving_gb300 as moe
from kv_helpers import DEV
from test_gpu_kv_evict import check, make

pytestmark = pytest.mark.gpu


def row_vecs(c):
    return c.pages[0, 0, 0].numel() * c.pages.element_size() // 16


def is_wide(c, n):
    """The call's rule: enough slices of 128 bytes for every SM."""
    return n * c.pages.shape[0] * -(-row_vecs(c) // 8) >= torch.cuda.get_device_properties(DEV).multi_processor_count


CASES = [
    # rank, rope, four, sequences, layers, 16-byte vectors of a row left for the last CTA
    (512, 64, True, 16, 3, 2),
    (512, 64, False, 12, 2, 0),
    (512, 16, False, 12, 2, 2),
    (512, 8, False, 18, 1, 1),
    (256, 32, True, 40, 2, 5),
    (488, 0, False, 10, 2, 5),
    (96, 24, False, 50, 2, 7),
]


@pytest.mark.parametrize("shared", [0, 3])
@pytest.mark.parametrize("rank,rope,four,n,layers,left", CASES)
def test_rows_of_all_widths(rank, rope, four, n, layers, left, shared):
    lens = [300 + (i * 131) % 700 for i in range(n)]
    c, w = make(lens, 64, layers, rank, rope, seed=rank + rope, shared_blocks=shared, four=four)
    assert is_wide(c, n) and row_vecs(c) % 8 == left
    check(c, w, list(range(n))[::-1], 320, 3, 40)


@pytest.mark.parametrize("page,budget,recent,shared", [(16, 100, 0, 0), (128, 500, 499, 2), (32, 999, 30, 5)])
def test_pages_and_budgets(page, budget, recent, shared):
    lens = [max(shared * page, (i * 211) % 1200) for i in range(20)]
    c, w = make(lens, page, 2, 512, 64, seed=page, shared_blocks=shared, four=True)
    assert is_wide(c, 20)
    check(c, w, list(range(20)), budget, 1, recent)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("shared", [0, 4])
def test_past_the_weights_in_registers(four, shared):
    """8192 tokens and one more are the border; one sequence goes far beyond it."""
    lens = [8192, 8193, 20001, 8500] + [700 + 13 * i for i in range(12)]
    c, w = make(lens, 64, 3, 512, 64, seed=7, shared_blocks=shared, four=four)
    assert is_wide(c, 16)
    check(c, w, list(range(16)), 600, 4, 100)


def test_few_go_and_most_go():
    lens = [1000] * 20
    for budget, recent in ((999, 10), (1, 0), (2, 1)):
        c, w = make(lens, 16, 2, 512, 64, seed=budget, four=True)
        assert is_wide(c, 20)
        check(c, w, list(range(20)), budget, 0, recent)


def test_refused_entries():
    lens = [200 + 10 * i for i in range(20)]
    c, w = make(lens, 16, 3, 512, 64, seed=5, four=True)
    seqs = list(range(20))
    seqs[3], seqs[7], seqs[11] = 0, -1, 99                   # a repeat and two ids out of range
    c.table[5, 4] = -1
    assert is_wide(c, 16)
    check(c, w, seqs, 64, 2, 8, bits=moe.MOE_DEV_ERR_BAD_SEQ | moe.MOE_DEV_ERR_BAD_PAGE)
