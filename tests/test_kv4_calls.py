"""Host side of the 4-bit cache's calls, without a GPU."""

import block_causal_streaming_sa_b200 as sa


def test_a_call_that_needs_no_workspace_asks_for_none():
    cache = sa.QuantKVCache.__new__(sa.QuantKVCache)  # nothing allocated yet
    cache._workspaces, cache._sizes = [], {}
    assert cache._work("none", lambda: 0, None) == (0, 0)
    assert cache._workspaces == []
