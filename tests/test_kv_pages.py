"""Page numbers of cache slots over the whole allowed range: slots up to 2^31 - 1, every
page size. The kernels divide by multiplication; the same function runs here on the host."""
import os

import pytest


@pytest.fixture(scope="module")
def L():
    from routing_q4_grouped_gb300 import build, moeq4
    if not os.path.exists(moeq4.LIB_PATH):
        build.build()
    return moeq4


@pytest.mark.parametrize("first", range(16, 4097, 16 * 16))
def test_page_of_a_slot(L, first):
    for P in range(first, min(first + 16 * 16, 4097), 16):
        last = (2 ** 31 - 1) // P                        # the last page, perhaps in part
        pages = {0, 1, 2, 3, last - 1, last}
        for e in range(2, 31):                           # either side of every power of two
            pages |= {max(0, (1 << e) // P + d) for d in (-1, 0, 1)} | {(1 << e) - 1, 1 << e, (1 << e) + 1}
        for page in pages:
            for slot in (page * P, page * P + 15, page * P + P // 2, page * P + P - 16, page * P + P - 1):
                if slot < 2 ** 31:
                    assert L.moe_debug_kv_page(P, slot) == slot // P, (P, slot)


def test_page_of_no_slot(L):
    assert L.moe_debug_kv_page(16, -1) == L.moe_debug_kv_page(24, 0) == L.moe_debug_kv_page(8192, 0) == -1
