"""Page plans and shared-prefix attention without a GPU: refusals of the C ABI and the binding, and the 64-bit
definitions that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import prefix_ref as R
import serving_ref as S


@pytest.fixture(scope="module")
def lib():
    import os

    import indexer_routed_sparse_gb300 as irs

    if not os.path.exists(irs.LIB_PATH):
        from indexer_routed_sparse_gb300 import build

        build.build()
    return irs.lib()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(1 << 20)
    p.keep = buf
    return ctypes.addressof(buf) + (256 - ctypes.addressof(buf) % 256) % 256


def _refused(lib, st, word):
    assert st == 2, lib.irs_last_error()
    assert word in lib.irs_last_error(), lib.irs_last_error()


def _plan(lib, p, **kw):
    at = {n: p + 4096 * i for i, n in enumerate(("lens", "new", "table", "free", "count", "cu", "pl", "cu_new", "pos", "slots",
                                                 "after", "left"))}
    a = dict(at, B=4, ts=8, mp=8, ps=16, nf=9, P=2, tokens=6)
    a.update({n: (at[x] if isinstance(x, str) else x) for n, x in kw.items()})
    return lib.irs_paged_plan(a["lens"], a["new"], a["B"], a["table"], a["ts"], a["mp"], a["ps"], a["free"], a["nf"], a["count"],
                              a["cu"], a["pl"], a["P"], a["tokens"], a["cu_new"], a["pos"], a["slots"], a["after"], a["left"],
                              None, None)


@pytest.mark.parametrize("kw,word", [
    (dict(B=0), b"sizes"), (dict(P=-1), b"sizes"), (dict(tokens=-1), b"sizes"), (dict(nf=-1), b"sizes"), (dict(mp=0), b"pool"),
    (dict(ps=0), b"pool"), (dict(mp=1 << 20, ps=1 << 11, ts=1 << 20), b"2^30"), (dict(ts=7), b"table_stride"),
    (dict(lens=None), b"NULL"), (dict(new=None), b"NULL"), (dict(table=None), b"NULL"), (dict(free=None), b"NULL"),
    (dict(count=None), b"NULL"), (dict(cu=None), b"NULL"), (dict(pl=None), b"NULL"), (dict(cu_new=None), b"NULL"),
    (dict(pos=None), b"NULL"), (dict(slots=None), b"NULL"), (dict(after=None), b"NULL"), (dict(left=None), b"NULL"),
    (dict(after="lens"), b"overlaps an input"), (dict(left="count"), b"overlaps an input"), (dict(pos="new"), b"overlaps an input"),
    (dict(table="free"), b"overlaps an input"), (dict(pos="slots"), b"outputs overlap"), (dict(cu_new="table"), b"outputs overlap"),
])
def test_plan_refusals(lib, p, kw, word):
    _refused(lib, _plan(lib, p, **kw), word)


def _prefix(lib, p, decode, **kw):
    a = dict(q=p, kc=p, vc=p, table=p, ts=8, mp=8, np=9, ps=16, lens=p, cu=p, pl=p, P=2, oo=None, ol=None, T=2, Hq=4, Hkv=2,
             Dqk=128, Dv=128, scale=0.1, out=p + 8192, lse=None, ws=p, wb=1 << 30, st=128)
    a.update(kw)
    head = (a["q"], 512, a["st"], a["kc"], 4096, 256, 128, a["vc"], 4096, 256, 128, a["table"], a["ts"], a["mp"], a["np"], a["ps"])
    tail = (a["T"], a["Hq"], a["Hkv"], a["Dqk"], a["Dv"], a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None, None)
    if decode:
        return lib.irs_shared_prefix_gqa_attn_decode(*head, a["lens"], a["cu"], a["pl"], a["P"], *tail)
    return lib.irs_shared_prefix_gqa_attn_fwd(*head, a["cu"], a["pl"], a["P"], a["oo"], a["ol"], *tail)


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("kw,word", [
    (dict(Hq=5), b"multiple"), (dict(Hkv=0), b"sizes"), (dict(T=-1), b"sizes"), (dict(P=-1), b"sizes"), (dict(P=0), b"one group"),
    (dict(Hq=258), b"128 query heads"), (dict(Dqk=256), b"Dqk"), (dict(Dqk=96), b"Dqk"), (dict(Dv=192), b"Dv"), (dict(Dv=256), b"Dv"),
    (dict(scale=0.0), b"scale"), (dict(scale=math.nan), b"scale"), (dict(ts=2), b"table_stride"), (dict(ps=0), b"pool"),
    (dict(mp=1 << 20, ps=1 << 11, ts=1 << 20), b"2^30"), (dict(q=None), b"NULL"), (dict(out=None), b"NULL"), (dict(ws=None), b"NULL"),
    (dict(cu=None), b"NULL"), (dict(pl=None), b"NULL"), (dict(kc=None), b"NULL"), (dict(vc=8), b"16-byte"), (dict(q=8), b"16-byte"),
    (dict(ws=16), b"256-byte"), (dict(wb=16), b"too small"), (dict(st=4), b"multiples of 8"), (dict(st=-128), b"multiples of 8"),
    (dict(out=512), b"out overlaps q"),
])
def test_attention_refusals(lib, p, decode, kw, word):
    kw = {n: (p + x if n in ("ws", "q", "vc", "out") and x else x) for n, x in kw.items()}
    _refused(lib, _prefix(lib, p, decode, **kw), word)


def test_attention_refusals_of_one_form(lib, p):
    _refused(lib, _prefix(lib, p, True, lens=None), b"NULL")
    _refused(lib, _prefix(lib, p, True, T=1 << 23), b"2^24")
    _refused(lib, _prefix(lib, p, True, Hq=64 * 1024, Hkv=1024), b"1024")
    _refused(lib, _prefix(lib, p, False, Hq=1025, Hkv=1025), b"1024")
    _refused(lib, _prefix(lib, p, False, T=1 << 30), b"2^31")
    _refused(lib, _prefix(lib, p, False, oo=p), b"come together")
    _refused(lib, _prefix(lib, p, False, oo=p + 8, ol=p), b"16-byte")
    _refused(lib, _prefix(lib, p, False, oo=p + 8192 + 16, ol=p), b"row by other row")
    _refused(lib, _prefix(lib, p, False, oo=p + 16384, ol=p + 32768, lse=p + 32772), b"row by other row")


def test_attention_of_nothing_is_fine(lib, p):
    assert _prefix(lib, p, False, T=0) == 0 and _prefix(lib, p, True, T=0) == 0
    for name in ("fwd", "decode"):
        size = getattr(lib, f"irs_shared_prefix_gqa_attn_{name}_workspace_bytes")
        assert size(4, 2, 8, 2, 128) > 0 and size(4, 2, 7, 2, 128) == 0 and size(-1, 2, 8, 2, 128) == 0


def test_binding_refuses_other_types_shapes_and_cpu_tensors():
    import indexer_routed_sparse_gb300 as irs

    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    table = torch.zeros(4, 2, dtype=torch.int32)
    for x, e in ((q.float(), TypeError), (q, ValueError)):
        with pytest.raises(e):
            irs.shared_prefix_gqa_attn_fwd(x, pool, pool, table, i, i)
        with pytest.raises(e):
            irs.shared_prefix_gqa_attn_decode(x, pool, pool, table, i, i, i)
    for x, e in ((i.long(), TypeError), (i, ValueError), (None, TypeError)):
        with pytest.raises(e):
            irs.paged_plan(x, i, table, i, i, 16, 4)


# ---------------------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------------------
def test_reference_plan_by_hand():
    """Pages of 4. Request 0 holds 3 tokens and takes 2: one page more; request 1 is new and takes 5; request 2 is full of
    a prefix of 6 tokens that it shares with request 0's first page."""
    table, cu, pos, slots, lens, left = R.plan([3, 0, 6], [2, 5, 1], [[9, -1], [-1, -1], [-1, 8]], [1, 2, 3, 4, 5], 5, 4, 9,
                                               [0, 3], [6])
    assert table == [[9, 5], [4, 3], [9, 8]]
    assert cu == [0, 2, 7, 8] and pos == [3, 4, 0, 1, 2, 3, 4, 6, -1]
    assert slots == [39, 20, 16, 17, 18, 19, 12, 34, -1]
    assert lens == [5, 5, 7] and left == 2


def test_reference_join_equals_one_softmax():
    """Attention over two halves of the keys, joined, is attention over all of them; a half of nothing does not count."""
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(*s, generator=g).double() for s in ((5, 4, 16), (23, 2, 16), (23, 2, 8)))
    whole = R.attend(q, k, v, 0.25)
    for m in (0, 1, 11, 23):
        out, lse, _, _ = R.join(R.attend(q, k[:m], v[:m], 0.25), R.attend(q, k[m:], v[m:], 0.25))
        assert (out - whole[0]).abs().max() < 1e-12 and (lse - whole[1]).abs().max() < 1e-12


def test_reference_decode_is_the_paged_decode():
    """Shared or not, a sequence attends its whole table."""
    g = torch.Generator().manual_seed(2)
    kc, vc = (torch.randn(20, 4, 2, d, generator=g).to(torch.bfloat16) for d in (64, 128))
    q = torch.randn(3, 4, 64, generator=g).to(torch.bfloat16)
    table = torch.tensor([[0, 1, 2, 9, 9], [0, 1, 2, 3, 4], [0, 1, 5, 9, 9]], dtype=torch.int32)
    lens = [11, 20, 9]
    a = R.decode(q, kc, vc, table, lens, [0, 2, 3], [11, 3], 0.125)
    b = S.decode(q, kc, vc, table, lens, 0.125)
    assert (a[0] - b[0]).abs().max() < 1e-12 and (a[1] - b[1]).abs().max() < 1e-12
    c = R.fwd(q, kc, vc, table, [0, 1, 2, 3], [11, 20, 9], 0.125)
    assert (c[0] - b[0]).abs().max() < 1e-12
