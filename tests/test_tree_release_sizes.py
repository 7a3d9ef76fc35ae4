"""Tables so wide that the pages of the requests that a release takes together pass 32 bits."""
import pytest

import gated_delta_rule_33_gb300 as kda
from test_tree_boundary import INVALID, SHAPE, far


@pytest.fixture(scope="module")
def clib():
    kda.build()
    return kda.load()


def test_wide_tables_are_refused(clib):
    def release(B, max_pages, shares=far(50)):
        return clib.kda_page_release(far(0), far(1), far(200), max_pages, B, 1, 1 << 20, shares, far(60), 8, far(70), None)
    for B, max_pages in ((1024, 1 << 21), (5000, 1 << 21), (3, (1 << 31) // 3 + 1), (1, 2 ** 31 - 1), (2, 1 << 30)):
        want = SHAPE if min(B, 1024) * max_pages >= 1 << 31 else INVALID
        assert release(B, max_pages, shares=None) == want, (B, max_pages)
    assert release(1024, (1 << 21) - 1, shares=None) == INVALID   # fits: the missing array is what is refused
