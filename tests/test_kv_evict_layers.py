"""Eviction's limit on layers: a launch has a dimension for them (no GPU: refused before any launch)."""
import ctypes

import edge_moe_serving_gb300 as moe
from test_latent_workspace import cache


def test_more_layers_than_a_launch_has():
    for layers, refused in ((65535, False), (65536, True)):
        c = cache(n_layers=layers, n_pages=16, page_tokens=16, max_blocks=4)
        assert (moe.moe_kv_evict_workspace_size(c, 1) == 0) == refused
        status = moe.lib().moe_kv_evict(ctypes.byref(c), 256, 1, 256, 8, 0, 0, None, None, 0, None, None)
        assert status == (moe.MOE_ERR_UNSUPPORTED if refused else moe.MOE_ERR_WORKSPACE)
