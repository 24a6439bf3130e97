"""Workspaces of the absorbed attention over a 4-bit cache with long shared
prefixes, whose bf16 copy is the largest part of them (sizes alone, no GPU)."""
import pytest

import edge_moe_serving_gb300 as moe
from test_latent_workspace import cache

size = moe.moe_latent_decode_workspace_size


def room(B, Q, heads, shared, **k):
    """What a workspace for a 4-bit cache has beyond a bf16 cache's: the prefix's bf16 copy, if any."""
    return size(cache(reserved=moe.MOE_KV_FP4, **k), B, Q, heads, shared) - size(cache(**k), B, Q, heads, shared)


@pytest.mark.parametrize("shared", [1 << 20, 1 << 24, 1 << 27])
@pytest.mark.parametrize("heads,Q", [(128, 1), (128, 8)])
def test_a_longer_list_has_room_for_what_its_parts_expand(heads, Q, shared):
    """A list of more than 512 sequences is launched in parts, in one workspace: 600 are 512 and 88."""
    copy = shared * (512 + 64) * 2
    rooms = [room(B, Q, heads, shared, max_blocks=1 << 21) for B in (1, 88, 512, 600, 4096)]
    assert rooms[1] >= copy and all(a <= b for a, b in zip(rooms, rooms[1:])), rooms


def test_sizes_never_fall_up_to_the_longest_prefix():
    c = cache(reserved=moe.MOE_KV_FP4, max_blocks=1 << 21)
    for heads, Q in ((16, 1), (128, 8)):
        for B in (88, 512, 4096):
            sizes = [size(c, B, Q, heads, 1 << x) for x in range(6, 28)]
            assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("four", [0, 1])
def test_sizes_never_fall_at_the_end_of_int(four):
    """Longer than any cache's prefix: the call refuses it, the size is still that of the longest."""
    c = cache(reserved=four, page_tokens=16, n_pages=4096, max_blocks=1 << 21)
    sizes = [size(c, 4, 1, 128, 2 ** 31 - x) for x in (128, 64, 32, 16, 1)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:])), sizes
