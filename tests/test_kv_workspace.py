"""Workspace sizes of attention: 0 exactly where the call refuses the sizes, whatever they
are; no device needed."""
import ctypes
import os

import pytest

FAKE = 1 << 20      # aligned non-null, never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


def call(L, B, nq, Hq, Hkv, D, max_len, prefix, ws_bytes):
    cache = L.KVCacheC(FAKE, FAKE, 4, 16, Hkv, D, 8)
    a = L.KVAttnC(FAKE, Hq * D, D, FAKE, Hq * D, D, FAKE, FAKE, FAKE, B, nq, Hq, 1 << 30, max_len,
                  prefix, 0.1)
    return L.lib().moe_kv_attention(ctypes.byref(a), ctypes.byref(cache), FAKE, ws_bytes, None)


BIG = 2 ** 31 - 1
CASES = [
    (1, 1, 16, 2, 128, 777, 0), (64, 4, 32, 8, 64, 8192, 65536), (1, 4096, 16, 2, 128, 32768, 0),
    (1, 1, 1, 1, 64, 2 ** 30, 2 ** 30), (2 ** 24, 1, 1, 1, 64, 16, 0), (3, 2, 4, 2, 256, 0, 0),
    # refused: more query tokens, heads, tokens or work than the call takes
    (2 ** 24 + 1, 1, 1, 1, 64, 16, 0), (2 ** 12, 2 ** 12 + 1, 1, 1, 64, 16, 0),
    (1, 1, 65536, 1, 64, 16, 0), (1, 1, 4, 2, 64, 2 ** 30 + 1, 0), (1, 1, 4, 2, 64, 0, 2 ** 30 + 1),
    (2 ** 20, 16, 4096, 1, 64, 16, 0), (2 ** 20, 1, 64, 8, 64, 2 ** 20, 0), (1, 1, 2048, 2048, 64, 16, 0),
    (BIG, BIG, BIG, 1, 256, BIG, BIG), (BIG, BIG, BIG, BIG, 64, BIG, BIG), (BIG, 1, 16, 1, 64, 0, 1),
    (1, BIG, 65535, 1, 256, 2 ** 30, 0), (1, 1, 5, 2, 64, 16, 0), (1, 1, 4, 2, 96, 16, 0),
]


@pytest.mark.parametrize("sizes", CASES)
def test_size_is_zero_where_the_call_refuses(L, sizes):
    B, nq, Hq, Hkv, D, max_len, prefix = sizes
    n = L.moe_kv_attention_workspace_size(*sizes)
    # (no workspace at all: sizes that are allowed are refused for that alone)
    assert call(L, *sizes, 0) == (-2 if n == 0 else -3), (sizes, n)
    if n:
        assert call(L, *sizes, n - 1) == -3 and n < 1 << 50


def test_partial_results_cover_the_least(L):
    # a call that is cut at all writes a row of D values and a pair per query row and head
    assert L.moe_kv_attention_workspace_size(1, 1, 32, 8, 128, 131071) >= 32 * (128 * 4 + 8)
