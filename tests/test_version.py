"""A caller can tell a library that reads the cache's format from one that ignored the field (no GPU)."""
import ctypes

import edge_moe_serving_gb300 as moe
from test_latent_workspace import cache


def test_version_says_that_the_format_is_read():
    c = cache(reserved=7)                                   # no format: refused, where 1.0.0 did not look
    assert moe.lib().moe_kv_workspace_size(ctypes.byref(c), 4) == 0
    assert moe.moe_version() >= 110
