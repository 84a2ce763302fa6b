"""Where shared-prefix attention joins a prefix's part with others, on the GPU: prefixes whose scores are all -inf, and
results that take their other part's place in rows that runs' borders cut."""
import math

import pytest
import torch

import prefix_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def irs():
    import indexer_routed_sparse_gb300 as m

    m.lib()
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inputs(seed, rows, prefix, Hq, Hkv, Dqk, Dv, page=16):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)

    need = [-(-n // page) for n in prefix]
    cu, starts = [0], [0]
    for r, n in zip(rows, need):
        cu.append(cu[-1] + r)
        starts.append(starts[-1] + n)
    table = torch.zeros(len(rows), max(need + [1]), dtype=torch.int32, device=DEV)
    for i, n in enumerate(need):
        table[i, :n] = torch.arange(starts[i], starts[i] + n, device=DEV)
    kc, vc = (normal(starts[-1] + 1, page, Hkv, d) for d in (Dqk, Dv))
    own = (normal(cu[-1], Hq, Dv), torch.randn(cu[-1], Hq, generator=g, device=DEV) * 4)
    return normal(cu[-1], Hq, Dqk), kc, vc, table, cu, own


@pytest.mark.parametrize("n", [5, 150, 9000])
@pytest.mark.parametrize("Dv", [64, 128])
def test_prompts_a_prefix_of_minus_infinity_leaves_the_own_part(irs, n, Dv):
    """Softmax over both sets has no weight on the prefix; a row without any other finite score is 0 / 0."""
    q, kc, vc, table, cu, own = _inputs(n + Dv, [40], [n], 8, 2, 128, Dv)
    q.abs_().clamp_(min=0.01)
    kc[:] = 0
    kc[..., 0] = -math.inf
    own[1][::3] = -math.inf
    out, lse = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), _i32([n]), own=own)
    irs.check_device_errors(DEV)
    none = own[1] == -math.inf
    # weight 1 on the own part: its own bits
    assert torch.equal(out[~none], own[0][~none]) and torch.equal(lse[~none], own[1][~none])
    assert out[none].isnan().all() and lse[none].isnan().all()


@pytest.mark.parametrize("Hq,Hkv,Dqk,Dv", [(16, 2, 128, 128), (16, 2, 64, 64), (32, 2, 192, 128), (5, 1, 128, 64)])
def test_prompts_in_place_where_borders_cut_items(irs, Hq, Hkv, Dqk, Dv):
    """out and lse in own's place: rows of items that several runs share, and of a group whose prefix is empty."""
    rows, prefix = [700, 333, 900, 1], [3001, 0, 2500, 0]
    q, kc, vc, table, cu, own = _inputs(Hq + Dv, rows, prefix, Hq, Hkv, Dqk, Dv)
    out, lse = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), _i32(prefix), own=own)
    ref = R.fwd(q, kc, vc, table, cu, prefix, 1 / math.sqrt(Dqk), own)
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")
    for _ in range(5):
        a, b = own[0].clone(), own[1].clone()
        irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), _i32(prefix), own=(a, b), out=a, lse=b)
        assert torch.equal(a, out) and torch.equal(b, lse)
    irs.check_device_errors(DEV)
