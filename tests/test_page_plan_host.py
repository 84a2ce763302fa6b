"""The page plan's argument checks without a GPU, and its definition by hand."""
import os

import pytest

import plan_ref as R


@pytest.fixture(scope="module")
def lib():
    import indexer_routed_sparse_gb300 as irs

    if not os.path.exists(irs.LIB_PATH):
        from indexer_routed_sparse_gb300 import build

        build.build()
    return irs.lib()


def test_results_without_tokens_lie_over_nothing(lib):
    """positions and slots of no token reach over no byte, wherever they point: what is refused is free_left, over an input."""
    at = {n: (i + 1) << 20 for i, n in enumerate(("lens", "new", "table", "free", "count", "cu_new", "after"))}
    st = lib.irs_paged_plan(at["lens"], at["new"], 4, at["table"], 8, 8, 16, at["free"], 9, at["count"], None, None, 0, 0,
                            at["cu_new"], at["cu_new"] + 4, at["lens"] + 8, at["after"], at["count"], None, None)
    assert st == 2 and lib.irs_last_error() == b"an output overlaps an input"
    st = lib.irs_paged_plan(at["lens"], at["new"], 4, at["table"], 8, 8, 16, at["free"], 9, at["count"], None, None, 0, 0,
                            at["cu_new"], at["cu_new"] + 4, at["after"] + 8, at["after"], at["cu_new"] + 8, None, None)
    assert st == 2 and lib.irs_last_error() == b"outputs overlap"


def test_definition_by_hand():
    """Pages of 4, tables of 8 positions. The first of a group of three takes its prompt of 8 in two steps and gives the page
    that is full; the second, which holds it, and the third ask for more than a table reaches."""
    table, cu, pos, slots, lens, left, refused = R.plan([3, 8, 0, 4], [3, 1, 30, 1], [[9, -1], [7, 8], [-1] * 2, [6, -1]], [1, 2, 3], 3,
                                                        4, 9, [0, 3], [8])
    assert refused and left == 1
    assert table == [[9, 3], [9, 8], [-1, -1], [6, 2]]
    assert cu == [0, 3, 3, 3, 4] and lens == [6, 8, 0, 5]
    assert pos == [3, 4, 5, 4, -1, -1, -1, -1, -1] and slots == [39, 12, 13, 8, -1, -1, -1, -1, -1]
