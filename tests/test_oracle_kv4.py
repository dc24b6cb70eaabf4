"""The 4-bit cache's oracle, pinned to hand-computed values, and the refusals of the
sa_kv4_* calls that need no GPU."""

import ctypes

import numpy as np
import pytest
import torch

import block_causal_streaming_sa_b200 as sa
from oracle import kv4


def block(x):
    v, byte = kv4.quantise_blocks(x[None])
    return v[0], int(byte[0])


def test_scale_table_is_fp16_of_the_byte_shifted_by_seven():
    bits = (np.arange(227, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(bits, kv4.SCALES)
    assert kv4.SCALES[226] == 10240.0 and kv4.MAX_STORED == 61440.0


def test_scale_is_the_smallest_that_covers_the_block():
    for amax, scale in [(6.0, 1.0), (6.001, 1.125), (5.9, 1.0), (0.75, 0.125), (6.75, 1.125),
                        (2.0 ** -20, 2.0 ** -17), (61440.0, 10240.0), (1e9, 10240.0)]:
        x = np.zeros(16)
        x[3] = -amax
        v, byte = block(x)
        assert kv4.SCALES[byte] == scale, amax
    assert block(np.zeros(16))[1] == 0


def test_ties_go_to_the_even_code():
    x = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -5, .26, .74, 4.99, 5.01, 0])
    v, byte = block(x)
    assert kv4.SCALES[byte] == 1.0
    assert v.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4, .5, .5, 4, 6, 0]


def test_stored_values_are_exact_in_fp16_and_bf16():
    vals = np.unique(np.outer(kv4.MAGNITUDES, kv4.SCALES))
    t = torch.from_numpy(vals)
    assert torch.equal(t.half().double(), t) and torch.equal(t.bfloat16().double(), t)


def test_attention_of_uniform_scores_is_the_mean_and_empty_rows_are_zero():
    keys, vals = np.zeros((4, 8)), np.arange(32.0).reshape(4, 8)
    o, lse, p, _ = kv4.attend(np.ones((3, 8)), keys, vals, [4, 2, 0], 1.0)
    assert np.allclose(o[0], vals.mean(0)) and np.allclose(o[1], vals[:2].mean(0))
    assert np.all(o[2] == 0) and lse[2] == -np.inf and np.all(p[2] == 0)
    assert np.isclose(lse[0], np.log(4))


def test_eviction_keeps_the_heaviest_and_fills_holes_in_order():
    w = np.array([5, 1, 4, 1, 0, 9, 2, 1.0])
    pos = np.arange(8)
    # keep 4 of 8: 5, 9, 4, 2 stay; row 1 takes row 5, row 3 takes row 6
    assert kv4.rows_after_eviction(w, pos, 8, 4, 0, 0) == [0, 5, 2, 6]
    # ties (the three 1s) go to the lower row
    assert kv4.rows_after_eviction(w, pos, 8, 5, 0, 0) == [0, 1, 2, 5, 6]
    # the first two and the last two stay whatever they weigh
    assert kv4.rows_after_eviction(w, pos, 8, 5, 2, 2) == [0, 1, 5, 6, 7]
    # NaN goes first, even before -inf
    w = np.array([np.nan, -np.inf, 1, 2.0])
    assert kv4.rows_after_eviction(w, pos[:4], 4, 3, 0, 0) == [3, 1, 2]


# ------------------------------------------------------------------ refusals (no GPU needed)

def _cache(**kw):
    fields = dict(batch=1, kv_heads=2, head_dim=64, capacity=128)
    fields.update(kw)
    return sa.SaKv4Cache(**fields)


def test_workspace_sizes():
    assert sa.sa_kv4_attend_bytes(_cache(), 4, 3) > 0
    assert sa.sa_kv4_attend_bytes(_cache(), 4, 0) == 0
    assert sa.sa_kv4_evict_bytes(_cache()) > 0
    for bad in (dict(batch=0), dict(kv_heads=0), dict(head_dim=96), dict(capacity=100),
                dict(capacity=0), dict(batch=1 << 17)):
        assert sa.sa_kv4_attend_bytes(_cache(**bad), 4, 3) == 0, bad
        assert sa.sa_kv4_evict_bytes(_cache(**bad)) == 0, bad
    assert sa.sa_kv4_attend_bytes(_cache(), 3, 3) == 0  # heads not a multiple of kv_heads
    assert sa.sa_kv4_attend_bytes(_cache(), 4, -1) == 0
    assert sa.sa_kv4_attend_bytes(None, 4, 3) == 0 and sa.sa_kv4_evict_bytes(None) == 0


def test_null_and_host_buffers_are_refused():
    lib = sa.lib()
    rows = sa.SaRows()
    assert lib.sa_kv4_reset(None, None) == sa.SA_ERR_INVALID_ARG
    assert lib.sa_kv4_get_status(None, None) == sa.SA_ERR_INVALID_ARG
    c = _cache()
    for call in (lambda: sa.sa_kv4_reset(c), lambda: sa.sa_kv4_append(c, rows, rows, 0, 1),
                 lambda: sa.sa_kv4_read(c, 0, rows, rows, 0, 1),
                 lambda: sa.sa_kv4_attend(c, rows, rows, 0, 2, 1),
                 lambda: sa.sa_kv4_evict(c, 1)):
        with pytest.raises(sa.SaError) as e:  # buffers NULL
            call()
        assert e.value.status == sa.SA_ERR_INVALID_ARG
        assert "kv4: k_codes" in sa.last_error()
    mem = torch.zeros(1 << 16, dtype=torch.uint8)
    at = (mem.data_ptr() + 15) & ~15
    c = _cache(**{f: at for f, _ in sa.SaKv4Cache._fields_[4:]})
    with pytest.raises(sa.SaError) as e:
        sa.sa_kv4_reset(c)
    assert e.value.status == sa.SA_ERR_INVALID_ARG
    bad = _cache(**{f: at + 8 for f, _ in sa.SaKv4Cache._fields_[4:]})
    with pytest.raises(sa.SaError) as e:
        sa.sa_kv4_reset(bad)
    assert "16-byte aligned" in sa.last_error()
    assert ctypes.sizeof(sa.SaKv4Cache) == 16 + 8 * 8 and ctypes.sizeof(sa.SaRows) == 32


def test_a_cache_off_the_gpu_is_refused():
    with pytest.raises(ValueError, match="must be on a GPU"):
        sa.QuantKVCache(1, 2, 64, 128, device="cpu")


def test_sizes_at_the_limits():
    assert sa.sa_kv4_evict_bytes(_cache(capacity=1 << 26)) == 2 * (4 << 26)
    assert sa.sa_kv4_attend_bytes(_cache(capacity=1 << 26), 2, 1, True) > 2 * (8 << 26)
    for bad in (dict(capacity=(1 << 26) + 128), dict(kv_heads=1 << 16),
                dict(batch=1 << 15, kv_heads=1 << 10)):
        assert sa.sa_kv4_evict_bytes(_cache(**bad)) == 0, bad
        assert "too many" in sa.last_error()
    assert sa.sa_kv4_attend_bytes(_cache(), 2, (1 << 24) + 1) == 0
    assert sa.sa_kv4_attend_bytes(_cache(kv_heads=1), 65535, 1 << 20) == 0
