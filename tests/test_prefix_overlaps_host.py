"""Shared-prefix attention whose outputs or workspace lie over what it reads, or over one another, is refused by the
C ABI. No memory is touched: the addresses are numbers."""
import pytest

NAMES = ("q", "k_cache", "v_cache", "page_table", "cu", "prefix_lens", "cache_lens", "own_out", "own_lse", "out", "lse", "workspace")
AT = {n: (i + 1) << 32 for i, n in enumerate(NAMES)}
T, P, HQ, HKV, D, PAGES, PAGE, WIDTH = 5, 2, 4, 2, 128, 9, 16, 8
# the bytes that each reaches over
SIZE = {"q": T * HQ * D * 2, "k_cache": PAGES * PAGE * HKV * D * 2, "v_cache": PAGES * PAGE * HKV * D * 2, "cu": 4 * (P + 1),
        "prefix_lens": 4 * P, "cache_lens": 4 * T, "own_out": T * HQ * D * 2, "own_lse": T * HQ * 4, "out": T * HQ * D * 2,
        "lse": T * HQ * 4}


@pytest.fixture(scope="module")
def lib():
    import os

    import indexer_routed_sparse_gb300 as irs

    if not os.path.exists(irs.LIB_PATH):
        from indexer_routed_sparse_gb300 import build

        build.build()
    return irs.lib()


def _size(lib, name, decode):
    if name == "page_table":
        return 4 * WIDTH * (T if decode else P)
    if name == "workspace":
        return getattr(lib, f"irs_shared_prefix_gqa_attn_{'decode' if decode else 'fwd'}_workspace_bytes")(T, P, HQ, HKV, D)
    return SIZE[name]


def _call(lib, decode, at):
    a = dict(AT, **at)
    pool = (PAGE * HKV * D, HKV * D, D)
    head = (a["q"], HQ * D, D, a["k_cache"], *pool, a["v_cache"], *pool, a["page_table"], WIDTH, WIDTH, PAGES, PAGE)
    tail = (T, HQ, HKV, D, D, 0.1, a["out"], a["lse"], a["workspace"], 1 << 31, None, None)
    if decode:
        st = lib.irs_shared_prefix_gqa_attn_decode(*head, a["cache_lens"], a["cu"], a["prefix_lens"], P, *tail)
    else:
        st = lib.irs_shared_prefix_gqa_attn_fwd(*head, a["cu"], a["prefix_lens"], P, a["own_out"], a["own_lse"], *tail)
    assert st == 2, lib.irs_last_error()
    return lib.irs_last_error().decode()


def _pairs():
    for decode in (False, True):
        ins = [n for n in NAMES[:9] if n not in (("own_out", "own_lse") if decode else ("cache_lens",))]
        for o in NAMES[9:]:
            for i in ins:
                if (o, i) not in (("out", "q"), ("out", "own_out"), ("lse", "own_lse")):   # refused in other words
                    yield decode, o, i
        yield decode, "lse", "out"
        yield decode, "workspace", "out"
        yield decode, "workspace", "lse"


@pytest.mark.parametrize("decode,a,b", list(_pairs()))
def test_overlaps_are_refused(lib, decode, a, b):
    align = {"out": 16, "lse": 4, "workspace": 256}[a]
    size, mine = _size(lib, b, decode), _size(lib, a, decode)
    last = AT[b] + (size - 1) // align * align          # a starts at b's end, or ends at its start
    first = AT[b] - (mine - 1) // align * align
    for at in (AT[b], last, first):
        assert f"{a} overlaps {b}" in _call(lib, decode, {a: at})


@pytest.mark.parametrize("decode", [False, True])
def test_neighbours_are_not(lib, decode):
    """Whatever lies right before or behind out is not over it: what is refused is the workspace, which is."""
    for n in NAMES[:6]:
        for at in (AT["out"] - _size(lib, n, decode), AT["out"] + SIZE["out"]):
            if at % 16 == 0:
                assert _call(lib, decode, {n: at, "workspace": AT["lse"] - AT["lse"] % 256}) == "workspace overlaps lse"


def test_results_in_the_other_parts_place_are_fine(lib):
    """out over own_out and lse over own_lse, each at the same address: only the workspace is refused."""
    assert _call(lib, False, {"out": AT["own_out"], "lse": AT["own_lse"], "workspace": AT["q"]}) == "workspace overlaps q"
    assert "row by other row" in _call(lib, False, {"out": AT["own_out"] + 16})
    assert "row by other row" in _call(lib, False, {"lse": AT["own_lse"] + 4})
    assert _call(lib, False, {"lse": AT["own_out"]}) == "lse overlaps own_out"
