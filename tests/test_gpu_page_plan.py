"""The page plan where pages run short and where a group's first sequence does not hold its prefix, on the GPU,
against an allocator on the host."""
import pytest
import torch

import plan_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def irs():
    import indexer_routed_sparse_gb300 as m

    m.lib()
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _check(irs, lens, new, table, free, page, groups=None, prefix=None, count=None, tokens=None):
    """One plan, and the same again, equal to the definition in everything; returns the definition's results."""
    count = len(free) if count is None else count
    tokens = sum(max(m, 0) for m in new) if tokens is None else tokens
    ref = R.plan(lens, new, table, free, count, page, tokens, groups, prefix)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dt = _i32(table)
    gr = {} if groups is None else dict(cu_groups=_i32(groups), prefix_lens=_i32(prefix))
    for _ in range(2):
        got = irs.paged_plan(_i32(lens), _i32(new), dt, _i32(free), _i32([count]), page, tokens, err=err, **gr)
        assert dt.tolist() == ref[0]
        assert got.cu_new.tolist() == ref[1] and got.positions.tolist() == ref[2] and got.slots.tolist() == ref[3]
        assert got.cache_lens.tolist() == ref[4] and got.free_count.tolist() == [ref[5]]
    assert int(err) == (irs.DEVERR_PAGE if ref[6] else 0)
    return ref


def test_a_refused_first_sequence_takes_nothing_from_the_others(irs):
    """One free page for a first sequence that needs three: the others, which hold the prefix, keep their pages."""
    ref = _check(irs, [0, 40], [40, 1], [[-1, -1, -1], [7, 8, 9]], [3], 16, [0, 2], [32])
    assert ref[0][1] == [7, 8, 9] and ref[4] == [0, 41]
    # it holds one page already, and gives that one only
    ref = _check(irs, [16, 40, 0], [30, 1, 0], [[5, -1, -1], [7, 8, 9], [-1, -1, -1]], [3], 16, [0, 3], [32])
    assert ref[0][1] == [5, 8, 9]


@pytest.mark.parametrize("n,m,given", [(0, 20, 1), (20, 0, 1), (20, 1, 1), (20, 11, 1), (20, 12, 2), (31, 1, 2), (0, 32, 2), (15, 0, 0),
                                       (0, 15, 0), (0, 48, 2), (33, 0, 2)])
def test_pages_that_the_first_sequence_fills_in_part_are_not_given(irs, n, m, given):
    """A first sequence that takes its prompt by and by gives the pages that are full after the step."""
    row = [20, 21, 22][: -(-n // 16)]
    ref = _check(irs, [n, 40], [m, 1], [row + [-1] * (4 - len(row)), [7, 8, 9, -1]], [1, 2, 3, 4], 16, [0, 2], [32])
    assert ref[0][1] == ref[0][0][:given] + [7, 8, 9][given:] + [-1]


def test_a_refused_sequence_takes_no_pages_from_those_behind_it(irs):
    ref = _check(irs, [0, 16, 3, 15], [160, 1, 0, 40], [[-1] * 10, [9] + [-1] * 9, [8] + [-1] * 9, [7] + [-1] * 9], [1, 2, 3, 4, 5], 16)
    assert ref[4] == [0, 17, 3, 55] and ref[5] == 1 and ref[0][1][:2] == [9, 5] and ref[0][3][:4] == [7, 4, 3, 2]
    # refused ones between others, and one that finds none at all
    _check(irs, [0, 0, 0, 0, 0], [33, 16, 65, 16, 1], [[-1] * 5] * 5, [1, 2, 3, 4, 5], 16)
    # a follower whose first sequence is given its pages behind a refused one
    _check(irs, [0, 0, 40], [100, 40, 1], [[-1] * 7, [-1] * 7, [7, 8, 9] + [-1] * 4], [1, 2, 3], 16, [0, 1, 3], [96, 32])


def test_a_length_past_the_table_refuses_new_tokens_and_nothing_else(irs):
    """A sequence whose new tokens are refused for their number holds, gives and takes pages of a prefix as ever."""
    table = [[4, 5, 6], [-1, -1, 9], [-1, -1, 8], [-1, -1, -1]]
    ref = _check(irs, [40, 40, 40, 60], [20, 1, -3, 1], table, [1, 2], 16, [0, 4], [32])
    assert [r[:2] for r in ref[0]] == [[4, 5], [4, 5], [4, 5], [-1, -1]] and ref[4] == [40, 41, 40, 60]


def test_an_idle_first_sequence_gives_what_its_row_names(irs):
    """As the decode reads a prefix: through the first sequence's row, idle or not; entries below 0 are not given."""
    ref = _check(irs, [0, 40, 32], [0, 1, 20], [[3, 4, -1, -1], [-1, -1, 9, -1], [-1] * 4], [1, 2], 16, [0, 3], [32])
    assert ref[0] == [[3, 4, -1, -1], [3, 4, 9, -1], [3, 4, 2, 1]]
    ref = _check(irs, [0, 40], [0, 1], [[3, -1, -1], [7, 8, 9]], [1], 16, [0, 2], [32])
    assert ref[0][1] == [3, 8, 9]


@pytest.mark.parametrize("B,page,seed", [(1, 16, 0), (5, 16, 1), (7, 1, 2), (40, 16, 3), (257, 48, 4), (300, 4, 5), (1100, 16, 6),
                                         (3000, 1, 7)])
@pytest.mark.parametrize("groups", [0, 1, 6])
def test_plans_that_run_short(irs, B, page, seed, groups):
    """Ragged requests, idle and unknown ones among them, and pages for a third to all of them."""
    g = torch.Generator().manual_seed(seed * 10 + groups)

    def pick(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))

    width = max(2, 120 // page)
    reach = width * page
    for share in (0.0, 0.35, 0.7, 1.0):
        lens = [pick(0, reach * 3 // 4) if pick(0, 3) else 0 for _ in range(B)]
        new = [min(pick(0, 2 if pick(0, 2) else reach // 2), reach - n) if pick(0, 3) else 0 for n in lens]
        if B > 4:
            lens[B // 2], new[B // 3], lens[B - 1] = -1, -2, reach + 1
        held = [-(-n // page) if 0 <= n <= reach else 0 for n in lens]
        need = sum(-(-(n + m) // page) - h for n, m, h in zip(lens, new, held) if 0 <= n and m >= 0 and n + m <= reach)
        order = torch.randperm(sum(held) + need + 3, generator=g).tolist()
        table = [[-1] * width for _ in lens]
        at = 0
        for row, h in zip(table, held):
            row[:h] = order[at: at + h]
            at += h
        free = order[at:]
        cuts = prefix = None
        if groups:
            cuts = [0] + sorted(pick(0, B) for _ in range(groups))
            prefix = [pick(0, reach // 2) for _ in range(groups)]
        _check(irs, lens, new, table, free, page, cuts, prefix, count=int(share * len(free)), tokens=sum(max(m, 0) for m in new) + 5)


def test_sizes_past_32_bits_are_refused(irs):
    """Of 2^32 + 16 a C int keeps 16."""
    args = _i32([3]), _i32([1]), _i32([[0, -1]]), _i32([5]), _i32([1])
    for page, tokens in (((1 << 32) + 16, 1), (16, 1 << 40), (16, -1), (0, 1), (-16, 1)):
        with pytest.raises(ValueError):
            irs.paged_plan(*args, page, tokens)


@pytest.mark.parametrize("B", [31, 33, 64, 700, 2100])
@pytest.mark.parametrize("free", [0, 1, 7, 40, 300])
def test_many_that_find_too_few(irs, B, free):
    """Needs in cycles, falling, scattered and alike: refusals lie among those that fit."""
    for needs in ([1 + i % 5 for i in range(B)], [max(1, 60 - i) for i in range(B)], [1 + (i * 7919) % 60 for i in range(B)], [50] * B):
        _check(irs, [0] * B, needs, [[-1] * max(needs)] * B, list(range(free)), 1)
