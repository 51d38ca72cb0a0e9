"""Host-side refusals of the gated linear recurrence's and the paged attention's entries: every bad argument is answered
before the device is touched."""
from __future__ import annotations

import ctypes

import pytest

import __graft_entry__
from gated_delta_rule_sm_gb300 import _lib

BAD, UNSUP, WS = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_ERR_WORKSPACE
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


def p(addr):
    return ctypes.c_void_p(addr) if addr else None


# (no call here is valid: one that passed the checks would be launched on these addresses)
def gated_dims(**kw):
    f = dict(B=1, T=100, C=64, dtype=_lib.KDA_BF16, num_seqs=0, x_stride=0, g_stride=0, i_stride=0)
    f.update(kw)
    return _lib.GatedDims(**f)


G = dict(x=1 * MB, g=2 * MB, i=3 * MB, a=4 * MB, cu=0, s0=5 * MB, y=6 * MB, sT=7 * MB, saved=8 * MB, nsaved=MB, ws=9 * MB, nws=MB,
         dy=10 * MB, dsT=11 * MB, dx=12 * MB, dg=13 * MB, di=14 * MB, da=15 * MB, ds0=16 * MB, host=None)


def fwd(lib, dims=None, **kw):
    a = {**G, **kw}
    return lib.kda_gated_scan_fwd(ctypes.byref(dims or gated_dims()), p(a["x"]), p(a["g"]), p(a["i"]), p(a["a"]), p(a["cu"]), a["host"], p(a["s0"]),
                                  p(a["y"]), p(a["sT"]), p(a["saved"]), a["nsaved"], p(a["ws"]), a["nws"], None)


def bwd(lib, dims=None, **kw):
    a = {**G, **kw}
    return lib.kda_gated_scan_bwd(ctypes.byref(dims or gated_dims()), p(a["x"]), p(a["g"]), p(a["i"]), p(a["a"]), p(a["cu"]), a["host"], p(a["s0"]),
                                  p(a["dy"]), p(a["dsT"]), p(a["dx"]), p(a["dg"]), p(a["di"]), p(a["da"]), p(a["ds0"]), p(a["saved"]), a["nsaved"],
                                  p(a["ws"]), a["nws"], None)


def step(lib, dims=None, slots=0, n=4, s_in=5 * MB, s_out=5 * MB, **kw):
    a = {**G, **kw}
    return lib.kda_gated_step(ctypes.byref(dims or gated_dims(B=4, T=1)), p(a["x"]), p(a["g"]), p(a["i"]), p(a["a"]), p(slots), n, p(s_in), p(s_out),
                              p(a["y"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), BAD), (dict(T=0), BAD), (dict(C=0), BAD), (dict(dtype=7), BAD), (dict(x_stride=63), BAD), (dict(g_stride=-64), BAD),
    (dict(i_stride=1), BAD), (dict(B=1 << 16, T=1 << 16), UNSUP), (dict(x_stride=1 << 40), UNSUP), (dict(T=1 << 30, C=1 << 12), UNSUP),
])
def test_gated_shapes(lib, kw, code):
    dims = gated_dims(**kw)
    assert fwd(lib, dims) == code and bwd(lib, dims) == code
    for name in ("kda_gated_scan_fwd_workspace_size", "kda_gated_scan_bwd_workspace_size", "kda_gated_scan_saved_size"):
        assert getattr(lib, name)(ctypes.byref(dims)) == 0
    if not ({"T", "x_stride"} & set(kw)) or code == BAD and "T" not in kw:
        assert step(lib, gated_dims(**{"T": 1, **kw}), n=1 << 30) == code


def test_gated_pointers_offsets_and_workspaces(lib):
    for name in ("x", "g", "i", "a", "y"):
        assert fwd(lib, **{name: 0}) == BAD
        assert step(lib, **{name: 0}) == BAD
    for name in ("x", "g", "i", "a", "dy", "dx", "dg", "di", "da"):
        assert bwd(lib, **{name: 0}) == BAD
    host = _lib.host_offsets([0, 60, 100], 3)
    for call in (fwd, bwd):
        assert call(lib, host=host) == BAD                                               # a host copy alone
        assert call(lib, gated_dims(B=2, T=50, num_seqs=2), cu=MB) == BAD
        assert call(lib, gated_dims(num_seqs=0), cu=MB) == BAD
        for off in ([1, 60, 100], [0, 60, 99], [0, 101, 100]):
            assert call(lib, gated_dims(num_seqs=2), cu=17 * MB, host=_lib.host_offsets(off, 3)) == BAD
        assert call(lib, ws=0) == WS and call(lib, ws=9 * MB + 16) == WS and call(lib, nws=64) == WS
        need = lib.kda_gated_scan_saved_size(ctypes.byref(gated_dims()))
        assert need == 2 * 64 * 4
        assert call(lib, nsaved=need - 1) == WS and call(lib, saved=8 * MB + 16) == WS
    assert step(lib, gated_dims(B=4, T=2)) == BAD
    assert step(lib, n=3) == BAD and step(lib, slots=MB, n=0) == BAD and step(lib, s_in=0) == BAD and step(lib, s_out=0) == BAD


N = 100 * 64 * 2       # bytes of x


@pytest.mark.parametrize("kw", [
    dict(y=1 * MB + N - 2), dict(y=1 * MB - N + 2), dict(y=2 * MB), dict(y=3 * MB), dict(y=5 * MB), dict(y=7 * MB), dict(y=8 * MB),
    dict(sT=1 * MB), dict(sT=2 * MB), dict(sT=3 * MB + N - 8), dict(sT=5 * MB + 8), dict(sT=8 * MB), dict(saved=1 * MB), dict(saved=5 * MB),
])
def test_gated_results_over_inputs(lib, kw):
    assert fwd(lib, **kw) == BAD


def test_gated_in_place_wants_contiguous_inputs(lib):
    assert fwd(lib, gated_dims(x_stride=128), y=G["x"]) == BAD


@pytest.mark.parametrize("out", ["dx", "dg", "di", "da", "ds0"])
@pytest.mark.parametrize("at", ["x", "g", "i", "a", "s0", "dy", "dsT", "saved", "dx", "dg", "di", "da", "ds0"])
def test_gated_gradients_over_anything(lib, out, at):
    if out != at:
        assert bwd(lib, **{out: G[at]}) == BAD


@pytest.mark.parametrize("kw", [dict(x_stride=(1 << 25) + 8), dict(g_stride=(1 << 25) + 8), dict(i_stride=1 << 31), dict(C=(1 << 25) + 2)])
def test_gated_offsets_that_pass_32_bits(lib, kw):
    big = dict(nws=1 << 40, nsaved=1 << 40)
    assert fwd(lib, gated_dims(**kw), **big) == UNSUP and bwd(lib, gated_dims(**kw), **big) == UNSUP
    assert step(lib, gated_dims(B=4, T=1, **kw)) == UNSUP


@pytest.mark.parametrize("at", ["a", "cu"])
def test_gated_results_over_the_rates_or_the_offsets(lib, at):
    dims, cu = gated_dims(num_seqs=3), 20 * MB
    to = cu + 12 if at == "cu" else G["a"] + 252
    for out in ("y", "sT", "saved"):
        over = to if out != "saved" else (cu if at == "cu" else G["a"])
        assert fwd(lib, dims, cu=cu, **{out: over}) == BAD
    for out in ("dx", "dg", "di", "da", "ds0"):
        assert bwd(lib, dims, cu=cu, **{out: to}) == BAD


@pytest.mark.parametrize("kw", [
    dict(y=2 * MB), dict(y=3 * MB + 500), dict(y=1 * MB + 2), dict(y=4 * MB), dict(y=5 * MB), dict(y=20 * MB + 12), dict(s_out=1 * MB),
    dict(s_out=2 * MB), dict(s_out=3 * MB), dict(s_out=4 * MB), dict(s_out=5 * MB + 256), dict(s_out=6 * MB), dict(s_out=20 * MB + 12),
])
def test_gated_step_results_over_inputs(lib, kw):
    assert step(lib, slots=20 * MB, **kw) == BAD
    assert step(lib, gated_dims(B=4, T=1, x_stride=128), y=G["x"]) == BAD


# ------------------------------------------------------------------------------------------- pages


def attn_dims(**kw):
    f = dict(rows=2, tokens=20, Hq=4, Hkv=2, D=64, dtype=_lib.KDA_BF16, num_pages=8, page_tokens=16, table_rows=3, max_pages=4, window=0,
             q_stride=0, k_stride=0, v_stride=0)
    f.update(kw)
    return _lib.AttentionDims(**f)


A = dict(q=1 * MB, pool=2 * MB, table=3 * MB, lengths=4 * MB, seqs=5 * MB, cu=0, host=None, scale=0.1, out=6 * MB, lse=7 * MB, ws=1 << 30, nws=1 << 40,
         k=8 * MB, v=9 * MB)


def attend(lib, dims=None, **kw):
    a = {**A, **kw}
    return lib.kda_pages_attention(ctypes.byref(dims or attn_dims()), p(a["q"]), p(a["pool"]), p(a["table"]), p(a["lengths"]), p(a["seqs"]), p(a["cu"]),
                                   a["host"], a["scale"], p(a["out"]), p(a["lse"]), p(a["ws"]), a["nws"], None)


def append(lib, dims=None, **kw):
    a = {**A, **kw}
    return lib.kda_pages_append(ctypes.byref(dims or attn_dims()), p(a["pool"]), p(a["table"]), p(a["lengths"]), p(a["seqs"]), p(a["cu"]), a["host"],
                                p(a["k"]), p(a["v"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), BAD), (dict(tokens=0), BAD), (dict(tokens=21), BAD), (dict(Hkv=0), BAD), (dict(D=0), BAD), (dict(dtype=4), BAD),
    (dict(num_pages=0), BAD), (dict(page_tokens=0), BAD), (dict(table_rows=0), BAD), (dict(max_pages=0), BAD), (dict(window=-1), BAD),
    (dict(D=257), UNSUP), (dict(D=264), UNSUP), (dict(tokens=(1 << 30) + 2), UNSUP), (dict(max_pages=1 << 20, page_tokens=1 << 20), UNSUP),
    (dict(num_pages=1 << 30, page_tokens=1 << 8), UNSUP),
])
def test_attention_shapes(lib, kw, code):
    assert attend(lib, attn_dims(**kw)) == code and append(lib, attn_dims(**kw)) == code
    if kw != dict(tokens=21):            # (with offsets that is fine)
        assert lib.kda_pages_attention_workspace_size(ctypes.byref(attn_dims(**kw))) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=0), BAD), (dict(Hq=5), BAD), (dict(q_stride=255), BAD), (dict(q_stride=1 << 40), UNSUP),
])
def test_attention_heads_and_strides(lib, kw, code):
    assert attend(lib, attn_dims(**kw)) == code


@pytest.mark.parametrize("kw,code", [(dict(k_stride=127), BAD), (dict(v_stride=-1), BAD), (dict(k_stride=1 << 40), UNSUP)])
def test_append_strides(lib, kw, code):
    assert append(lib, attn_dims(**kw)) == code


def test_attention_pointers_offsets_and_workspace(lib):
    for name in ("q", "pool", "table", "lengths", "out"):
        assert attend(lib, **{name: 0}) == BAD
    for name in ("pool", "table", "lengths", "k", "v"):
        assert append(lib, **{name: 0}) == BAD
    host = _lib.host_offsets([0, 5, 20], 3)
    for call in (attend, append):
        assert call(lib, host=host) == BAD
        assert call(lib, attn_dims(rows=4), seqs=0) == BAD                   # more rows than the table has
        for off in ([1, 5, 20], [0, 5, 19], [0, 21, 20]):
            assert call(lib, cu=17 * MB, host=_lib.host_offsets(off, 3)) == BAD
    for scale in (float("nan"), float("inf")):
        assert attend(lib, scale=scale) == BAD
    assert attend(lib, ws=0) == WS and attend(lib, ws=(1 << 30) + 16) == WS and attend(lib, nws=64) == WS
    assert lib.kda_pages_attention_workspace_size(None) == 0


Q, POOL = 20 * 4 * 64 * 2, 8 * 2 * 2 * 16 * 64 * 2


@pytest.mark.parametrize("kw", [
    dict(out=1 * MB), dict(out=1 * MB + Q - 16), dict(out=2 * MB + POOL - 16), dict(out=7 * MB), dict(lse=1 * MB), dict(lse=2 * MB),
])
def test_attention_results_over_inputs(lib, kw):
    assert attend(lib, **kw) == BAD


@pytest.mark.parametrize("at", ["table", "lengths", "seqs", "cu"])
def test_results_over_what_names_the_pages(lib, at):
    cu = dict(cu=18 * MB)
    for out in ("out", "lse"):
        assert attend(lib, **cu, **{out: {**A, **cu}[at]}) == BAD
    assert append(lib, **{**cu, at: A["pool"] + POOL - 4}) == BAD


@pytest.mark.parametrize("kw", [dict(k=2 * MB), dict(v=2 * MB + POOL - 16), dict(v=2 * MB - 16)])
def test_append_from_the_pool_itself(lib, kw):
    assert append(lib, **kw) == BAD
