"""Rotary, paged-cache and window operators without a GPU: refusals of the C ABI and the
binding, rotary frequencies, and the 64-bit definitions the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import serving_ref as R


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
    buf = ctypes.create_string_buffer(1024)
    p.keep = buf
    return ctypes.addressof(buf) + (256 - ctypes.addressof(buf) % 256) % 256


def _refused(lib, st, word):
    assert st == 2, lib.irs_last_error()
    assert word in lib.irs_last_error(), lib.irs_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), b"sizes"), (dict(H=0), b"sizes"), (dict(D=100), b"multiple of 8"), (dict(n=24), b"multiple of 16"),
    (dict(n=-16), b"multiple of 16"), (dict(start=4), b"multiple of 8"), (dict(start=72), b"inside the head"),
    (dict(start=-8), b"inside the head"), (dict(layout=2), b"layout"), (dict(amp=math.nan), b"amplitude"),
    (dict(f=None), b"inv_freq"), (dict(x=None), b"NULL"), (dict(pos=None), b"NULL"), (dict(out=None), b"NULL"),
    (dict(xo=8), b"16-byte"), (dict(st=132), b"multiples of 8"), (dict(st=-128), b"multiples of 8"),
    (dict(same=True, ost=256), b"x's strides"),
])
def test_rope_refusals(lib, p, kw, word):
    a = dict(T=4, H=2, D=128, n=64, start=0, layout=0, amp=1.0, f=p, x=p, pos=p, out=p + 512, xo=0, st=128, ost=128, same=False)
    a.update(kw)
    x = None if a["x"] is None else a["x"] + a["xo"]
    out = x if a["same"] else a["out"]
    _refused(lib, lib.irs_rope(x, 256, a["st"], a["pos"], a["f"], a["T"], a["H"], a["D"], a["n"], a["start"], a["layout"],
                               a["amp"], 0, out, 256, a["ost"], None), word)


def _append(lib, p, **kw):
    a = dict(q=p, k=p, v=p, cu=p, T=4, B=2, Hq=4, Hkv=2, Dqk=128, Dv=128, table=p, ts=8, mp=8, np=9, ps=16, lens=p, f=p, n=64,
             start=0, layout=1, amp=1.0, kc=p, vc=p, qo=p + 512, ko=None, st=128)
    a.update(kw)
    s = a["st"]
    return lib.irs_paged_rope_append(a["q"], 512, s, a["k"], 256, 128, a["v"], 256, 128, a["cu"], a["T"], a["B"], a["Hq"],
                                     a["Hkv"], a["Dqk"], a["Dv"], a["table"], a["ts"], a["mp"], a["np"], a["ps"], a["lens"],
                                     a["f"], a["n"], a["start"], a["layout"], a["amp"], a["kc"], 4096, 256, 128, a["vc"],
                                     4096, 256, 128, a["qo"], 512, 128, a["ko"], 256, 128, None, None)


@pytest.mark.parametrize("kw,word", [
    (dict(B=0), b"sizes"), (dict(Hkv=0), b"sizes"), (dict(cu=None), b"cu_new"), (dict(Dv=100), b"Dv"), (dict(n=40), b"multiple of 16"),
    (dict(mp=0), b"pool"), (dict(ps=0), b"pool"), (dict(np=0), b"pool"), (dict(mp=1 << 20, ps=1 << 11, ts=1 << 20), b"2^30"),
    (dict(ts=7), b"table_stride"), (dict(kc=None), b"NULL"), (dict(lens=None), b"NULL"), (dict(q=None), b"NULL"),
    (dict(qo=None), b"NULL"), (dict(v=None), b"NULL"), (dict(kc=8), b"16-byte"), (dict(ko=24), b"16-byte"), (dict(st=130), b"multiples of 8"),
])
def test_append_refusals(lib, p, kw, word):
    kw = {n: (p + x if n in ("kc", "ko") and x else x) for n, x in kw.items()}
    _refused(lib, _append(lib, p, **kw), word)


def test_append_of_nothing_is_fine(lib, p):
    assert _append(lib, p, T=0) == 0


def _decode(lib, p, **kw):
    a = dict(q=p, kc=p, vc=p, table=p, ts=8, mp=8, np=9, ps=16, lens=p, route=None, rs=0, W=0, window=0, sinks=0, B=2, Hq=4,
             Hkv=2, Dqk=128, Dv=128, scale=0.1, out=p, lse=None, ws=p, wb=1 << 30, st=128)
    a.update(kw)
    return lib.irs_paged_gqa_attn_decode(a["q"], 512, a["st"], a["kc"], 4096, 256, 128, a["vc"], 4096, 256, 128, a["table"],
                                         a["ts"], a["mp"], a["np"], a["ps"], a["lens"], a["route"], a["rs"], a["W"],
                                         a["window"], a["sinks"], a["B"], a["Hq"], a["Hkv"], a["Dqk"], a["Dv"], a["scale"],
                                         a["out"], a["lse"], a["ws"], a["wb"], None, None)


@pytest.mark.parametrize("kw,word", [
    (dict(Hq=5), b"multiple"), (dict(Hkv=0), b"sizes"), (dict(Dqk=96), b"Dqk"), (dict(Dqk=320), b"Dqk"), (dict(Dv=192), b"Dv"),
    (dict(window=-1), b"window"), (dict(sinks=-1), b"sinks"), (dict(sinks=3), b"window or routes"), (dict(W=4), b"without routes"),
    (dict(route=256, W=0), b"routes need"), (dict(route=256, W=4, rs=3), b"routes need"), (dict(scale=0.0), b"scale"),
    (dict(scale=math.inf), b"scale"), (dict(ts=2), b"table_stride"), (dict(ps=0), b"pool"), (dict(q=None), b"NULL"),
    (dict(out=None), b"NULL"), (dict(ws=None), b"NULL"), (dict(ws=16), b"256-byte"), (dict(wb=16), b"too small"),
    (dict(st=4), b"multiples of 8"), (dict(B=1 << 23), b"2^24"), (dict(Hq=2000, Hkv=1025), b"multiple"), (dict(Hq=1025, Hkv=1025), b"1024"),
])
def test_decode_refusals(lib, p, kw, word):
    kw = {n: (p + x if n in ("ws", "route") and x else x) for n, x in kw.items()}
    _refused(lib, _decode(lib, p, **kw), word)


def test_decode_sizes(lib, p):
    assert _decode(lib, p, B=0) == 0
    assert lib.irs_paged_gqa_attn_decode_workspace_bytes(4, 8, 2, 128) > 0
    assert lib.irs_paged_gqa_attn_decode_workspace_bytes(4, 7, 2, 128) == 0


def _window(lib, p, bwd=False, **kw):
    a = dict(q=p, k=p, v=p, cu=p, ndocs=2, window=8, sinks=2, T=16, Hq=4, Hkv=2, Dqk=128, Dv=128, scale=0.1, out=p, lse=p, dout=p,
             dq=p, dk=p, dv=p, ws=p, wb=1 << 30, st=128)
    a.update(kw)
    head = (a["q"], 512, a["st"], a["k"], 256, 128, a["v"], 256, 128, a["cu"], a["ndocs"], a["window"], a["sinks"])
    sizes = (a["T"], a["Hq"], a["Hkv"], a["Dqk"], a["Dv"], a["scale"])
    if bwd:
        return lib.irs_window_gqa_attn_bwd(*head, a["out"], a["lse"], a["dout"], *sizes, a["dq"], a["dk"], a["dv"], a["ws"],
                                           a["wb"], None, None)
    return lib.irs_window_gqa_attn_fwd(*head, *sizes, a["out"], a["lse"], None, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,word", [
    (dict(Hq=5), b"multiple"), (dict(Hq=258), b"128 query heads"), (dict(Dqk=256), b"Dqk"), (dict(Dv=192), b"Dv"),
    (dict(window=0), b"window"), (dict(window=-3), b"window"), (dict(sinks=129), b"sinks"), (dict(sinks=-1), b"sinks"),
    (dict(scale=-1.0), b"scale"), (dict(T=-1), b"sizes"), (dict(ndocs=0), b"ndocs"), (dict(ndocs=17), b"ndocs"),
    (dict(q=None), b"NULL"), (dict(cu=None), b"NULL"), (dict(k=8), b"16-byte"), (dict(st=12), b"multiples of 8"),
    (dict(T=1 << 30, Hq=4), b"2^31"), (dict(out=None), b""),
])
def test_window_refusals(lib, p, bwd, kw, word):
    kw = {n: (p + x if n == "k" and x else x) for n, x in kw.items()}
    _refused(lib, _window(lib, p, bwd, **kw), word)


def test_window_backward_buffers(lib, p):
    _refused(lib, _window(lib, p, True, lse=None), b"NULL")
    _refused(lib, _window(lib, p, True, dk=p + 8), b"16-byte")
    _refused(lib, _window(lib, p, True, wb=8), b"too small")
    _refused(lib, _window(lib, p, True, ws=p + 16), b"256-byte")
    assert _window(lib, p, True, T=0) == 0 and _window(lib, p, False, T=0) == 0
    assert lib.irs_window_gqa_attn_bwd_workspace_bytes(1000, 8, 2, 128, 128, 3, 64, 4) >= 1000 * 8 * 4
    assert lib.irs_window_gqa_attn_bwd_workspace_bytes(1000, 7, 2, 128, 128, 3, 64, 4) == 0


def test_binding_refuses_other_types_and_cpu_tensors():
    import indexer_routed_sparse_gb300 as irs

    b = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    table = torch.zeros(4, 2, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64)
    for x, e in ((b.float(), TypeError), (b, ValueError)):
        with pytest.raises(e):
            irs.rope(x, i, f)
        with pytest.raises(e):
            irs.paged_rope_append(x, x, x, pool, pool, table, i, f)
        with pytest.raises(e):
            irs.paged_gqa_attn_decode(x, pool, pool, table, i)
        with pytest.raises(e):
            irs.window_gqa_attn_fwd(x, x, x, i, 4)
        with pytest.raises(e):
            irs.window_gqa_attn_bwd(x, x, x, i, 4, b, b, b)


def test_rope_frequencies():
    import indexer_routed_sparse_gb300 as irs

    f, amp = irs.rope_frequencies(128)
    assert f.dtype == torch.float64 and f.shape == (64,) and amp == 1.0
    assert f[0] == 1.0 and torch.allclose(f, 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64), rtol=1e-14)
    lin, _ = irs.rope_frequencies(128, scaling="linear", factor=4.0)
    assert torch.equal(lin, f / 4)
    base, _ = irs.rope_frequencies(128, scaling="base", factor=4.0)
    assert base[0] == 1.0 and abs(base[-1] / (f[-1] / 4) - 1) < 1e-12       # the slowest pair slows by the factor
    parts, amp = irs.rope_frequencies(128, scaling="by_parts", factor=4.0, trained_len=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], f[turns >= 32]) and torch.equal(parts[turns <= 1], f[turns <= 1] / 4)
    assert (parts <= f).all() and (parts >= f / 4).all() and abs(amp - (0.1 * math.log(4) + 1)) < 1e-15
    for kw in (dict(rope_dims=20), dict(base=-1.0), dict(factor=0.5, scaling="linear"), dict(factor=2.0),
               dict(scaling="other"), dict(scaling="by_parts", factor=2.0)):
        with pytest.raises(ValueError):
            irs.rope_frequencies(**{**dict(rope_dims=64), **kw})


def test_reference_rotation_keeps_length_and_inverts():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20, 2, 64, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 10**6, (20,), generator=g)
    f = 10000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)
    for layout in ("half", "interleaved"):
        y, _ = R.rotate(x, pos, f, layout, 16, 1.0)
        assert torch.allclose(y.norm(dim=-1), x.double().norm(dim=-1), rtol=1e-12)
        back, _ = R.rotate(y, pos, f, layout, 16, 1.0, transpose=True)
        assert torch.allclose(back, x.double(), atol=1e-12)


def test_reference_window_equals_autograd_and_differences():
    g = torch.Generator().manual_seed(1)
    T, Hq, Hkv, D, window, sinks, scale = 40, 4, 2, 16, 7, 3, 0.25
    cu = torch.tensor([0, 11, 40], dtype=torch.int32)
    q, k, v, do = (torch.randn(T, h, D, generator=g, dtype=torch.float64) for h in (Hq, Hkv, Hkv, Hq))
    out, lse, _, _ = R.window_fwd(q, k, v, cu, window, sinks, scale)
    ours = R.window_bwd(q, k, v, cu, window, sinks, scale, out, lse, do)
    loss, grads = R.window_loss_grads(q, k, v, cu, window, sinks, scale, do)
    assert torch.allclose((out * do).sum(), loss, rtol=1e-12)
    for name, want in zip(("dq", "dk", "dv"), grads):
        assert torch.allclose(ours[name][0], want, atol=1e-10), name
    for i, name in enumerate(("dq", "dk", "dv")):            # and central differences along a direction
        d = torch.randn(*(q, k, v)[i].shape, generator=g, dtype=torch.float64)
        ends = []
        for s in (1e-5, -1e-5):
            args = [q, k, v]
            args[i] = args[i] + s * d
            ends.append((R.window_fwd(*args, cu, window, sinks, scale)[0] * do).sum())
        assert abs((ends[0] - ends[1]) / 2e-5 - (ours[name][0] * d).sum()) < 1e-6


def test_reference_decode_is_the_windows_last_row():
    g = torch.Generator().manual_seed(2)
    n, page = 37, 8
    k, v = torch.randn(n, 2, 64, generator=g).to(torch.bfloat16), torch.randn(n, 2, 64, generator=g).to(torch.bfloat16)
    q = torch.randn(n, 4, 64, generator=g).to(torch.bfloat16)
    table = torch.randperm(5, generator=g).to(torch.int32)[None]
    kc, vc = torch.full((5, page, 2, 64), math.nan, dtype=torch.bfloat16), torch.full((5, page, 2, 64), math.nan, dtype=torch.bfloat16)
    for t in range(n):
        kc[table[0, t // page], t % page], vc[table[0, t // page], t % page] = k[t], v[t]
    for window, sinks in ((0, 0), (9, 3)):
        w = R.window_fwd(q, k, v, torch.tensor([0, n]), window or n, sinks, 0.125)
        d = R.decode(q[-1:], kc, vc, table, torch.tensor([n]), 0.125, window, sinks)
        assert torch.allclose(w[0][-1], d[0][0], atol=1e-14) and torch.allclose(w[1][-1], d[1][0], atol=1e-14)
    r = R.decode(q[-1:], kc, vc, table, torch.tensor([n]), 0.125, routes=torch.arange(n)[None])
    assert torch.allclose(r[0], R.decode(q[-1:], kc, vc, table, torch.tensor([n]), 0.125)[0], atol=1e-14)


@pytest.mark.parametrize("T,ndocs,window,sinks", [(131072, 1000, 128, 128), (65536, 4000, 8, 64), (65536, 1, 1, 1),
                                                  (1 << 20, 1 << 19, 1, 128), (32768, 11, 512, 4), (50, 50, 1, 128), (9000, 3, 8000, 128)])
def test_window_backward_workspace_grows_with_tokens(lib, T, ndocs, window, sinks):
    """However many documents there are: D and the marks of keys, and FP32 rows for 3 of 8 keys at most."""
    Hq, Hkv, Dqk, Dv = 16, 8, 192, 128
    got = lib.irs_window_gqa_attn_bwd_workspace_bytes(T, Hq, Hkv, Dqk, Dv, ndocs, window, sinks)
    assert got <= 4 * T * Hq + T * Hkv // 8 + 12 * ndocs + 4096 + 3 * T // 8 * Hkv * (Dqk + Dv) * 4


@pytest.mark.parametrize("ot,oh", [(0, 128), (256, 0), (64, 128), (256, 120)])
def test_rope_refuses_outputs_that_overlap_themselves(lib, p, ot, oh):
    """Tokens or heads that share a row of the output would be written over one another in any order."""
    _refused(lib, lib.irs_rope(p, 256, 128, p, p, 4, 2, 128, 64, 0, 0, 1.0, 0, p + 512, ot, oh, None), b"overlap")


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("stride", [0, 64])
def test_append_refuses_caches_that_overlap_themselves(lib, p, which, stride):
    st = [4096, 256, 128, 4096, 256, 128]
    st[which] = stride
    _refused(lib, lib.irs_paged_rope_append(None, 0, 0, p, 256, 128, p, 256, 128, p, 4, 2, 0, 2, 128, 128, p, 8, 8, 9, 16, p, p, 64,
                                            0, 1, 1.0, p, *st[:3], p, *st[3:], None, 0, 0, None, 0, 0, None, None), b"overlap")


@pytest.mark.parametrize("qo,ko,word", [((0, 128), (256, 128), b"overlap"), ((512, 0), (256, 128), b"overlap"),
                                        ((512, 128), (0, 128), b"overlap"), ((512, 128), (256, 0), b"overlap"),
                                        ((512, 128), (512, 128), b"k's strides")])
def test_append_refuses_outputs_that_overlap(lib, p, qo, ko, word):
    k_out = p if word == b"k's strides" else p + 256
    _refused(lib, lib.irs_paged_rope_append(p, 512, 128, p, 256, 128, p, 256, 128, p, 4, 2, 4, 2, 128, 128, p, 8, 8, 9, 16, p, p, 64,
                                            0, 1, 1.0, p, 4096, 256, 128, p, 4096, 256, 128, p + 512, *qo, k_out, *ko, None, None), word)


@pytest.mark.parametrize("bwd,kw", [(False, dict(out=q)) for q in "qkv"] + [
    (True, {o: i}) for o in ("dq", "dk", "dv") for i in ("q", "k", "v", "dout")] + [(True, dict(dk="dq")), (True, dict(dv="dk"))])
@pytest.mark.parametrize("by", [0, 256])
def test_window_refuses_outputs_over_inputs(lib, p, bwd, kw, by):
    """Rows that are computed again, and dk and dv, read inputs after the first outputs are written. One output lies at
    or just behind the start of another tensor; all the others are apart."""
    at = {n: p + (i << 20) for i, n in enumerate(("q", "k", "v", "cu", "out", "lse", "dout", "dq", "dk", "dv", "ws"))}
    at.update({o: at[i] + by for o, i in kw.items()})
    _refused(lib, _window(lib, p, bwd, **at), b"overlap")


@pytest.mark.parametrize("kw", [dict(by=256), dict(Dqk=64), dict(Dv=64)])
def test_window_backward_refuses_dq_over_other_rows_of_out(lib, p, kw):
    at = {n: p + (i << 20) for i, n in enumerate(("q", "k", "v", "cu", "out", "lse", "dout", "dk", "dv", "ws"))}
    kw = dict(kw)
    _refused(lib, _window(lib, p, True, dq=at["out"] + kw.pop("by", 0), **kw, **at), b"overlaps out")
