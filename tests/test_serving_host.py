"""Host-side refusals of the serving entries: every bad argument is answered before the device is touched."""
from __future__ import annotations

import ctypes

import pytest
import torch

import __graft_entry__
import gated_delta_rule_sm_gb300 as kda
from gated_delta_rule_sm_gb300 import _lib

BAD, UNSUP, WS = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


def p(addr=4096):
    return ctypes.c_void_p(addr) if addr else None


def ssm_dims(**kw):
    f = dict(B=1, T=100, H=4, G=2, N=64, P=64, dtype=_lib.KDA_BF16, num_seqs=0, x_stride=0, b_stride=0, c_stride=0,
             dt_stride=0)
    f.update(kw)
    return _lib.SsmDims(**f)


def ssm_fwd(lib, dims, x=4096, y=4096, cu=None, host=None, ws=None, nb=0):
    return lib.kda_ssm_fwd(ctypes.byref(dims), p(x), p(), p(), p(), p(), p(), None, cu, host, None, p(y), None, ws, nb,
                           None)


def ssm_step(lib, dims, slots=None, n=1, s_in=4096, s_out=4096):
    return lib.kda_ssm_step(ctypes.byref(dims), p(), p(), p(), p(), p(), p(), None, slots, n, p(s_in), p(s_out), p(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), BAD), (dict(T=0), BAD), (dict(H=0), BAD), (dict(G=0), BAD), (dict(H=5), BAD), (dict(N=0), BAD),
    (dict(P=0), BAD), (dict(dtype=5), BAD), (dict(x_stride=255), BAD), (dict(b_stride=100), BAD),
    (dict(c_stride=-8), BAD), (dict(dt_stride=3), BAD), (dict(N=257), UNSUP), (dict(P=257), UNSUP),
    (dict(B=1 << 16, T=1 << 16), UNSUP), (dict(x_stride=1 << 40), UNSUP),
])
def test_scan_and_step_shapes(lib, kw, code):
    assert ssm_fwd(lib, ssm_dims(**kw)) == code
    if "T" not in kw and kw != dict(x_stride=1 << 40):     # with one row that stride is fine
        assert ssm_step(lib, ssm_dims(**{"T": 1, **kw}), n=1 << 30) == code
    assert lib.kda_ssm_fwd_workspace_size(ctypes.byref(ssm_dims(**kw))) == 0


def test_scan_pointers_offsets_and_workspace(lib):
    assert lib.kda_ssm_fwd(None, *[p()] * 6, None, None, None, None, p(), None, None, 0, None) == BAD
    assert ssm_fwd(lib, ssm_dims(), x=0) == BAD
    assert ssm_fwd(lib, ssm_dims(), y=0) == BAD
    host = _lib.host_offsets([0, 60, 100], 3)
    assert ssm_fwd(lib, ssm_dims(), host=host) == BAD                            # a host copy alone
    assert ssm_fwd(lib, ssm_dims(B=2, num_seqs=2), cu=p()) == BAD                # packed needs B == 1
    assert ssm_fwd(lib, ssm_dims(num_seqs=0), cu=p()) == BAD
    for bad in ([1, 60, 100], [0, 60, 99], [0, 101, 100]):
        assert ssm_fwd(lib, ssm_dims(num_seqs=2), cu=p(), host=_lib.host_offsets(bad, 3)) == BAD
    dims = ssm_dims(num_seqs=2)
    need = lib.kda_ssm_fwd_workspace_size(ctypes.byref(dims))
    assert need > 0
    assert ssm_fwd(lib, dims, cu=p(), host=host) == WS
    assert ssm_fwd(lib, dims, cu=p(), host=host, ws=p(4096 + 16), nb=need) == WS
    assert lib.kda_ssm_fwd_workspace_size(None) == 0


def test_step_pools(lib):
    one = ssm_dims(B=4, T=1)
    assert ssm_step(lib, ssm_dims(B=4, T=2), n=4) == BAD
    assert ssm_step(lib, one, n=3) == BAD                 # no slots: a slot per row
    assert ssm_step(lib, one, slots=p(), n=0) == BAD
    assert ssm_step(lib, one, n=4, s_in=0) == BAD
    assert ssm_step(lib, one, n=4, s_out=0) == BAD


def decode(lib, B=2, T=1, H=4, K=64, V=64, Hk=0, gate=0, dtype=0, lb=-5.0, scale=0.1, n=2, slots=None, q=4096, st=4096):
    dims = _lib.KdaDims(B, T, H, K, V, dtype, 0, Hk, gate)
    return lib.kda_decode_step(ctypes.byref(dims), p(q), *[p()] * 6, scale, lb, slots, n, p(st), p(st), p(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=2), BAD), (dict(B=0), BAD), (dict(H=0), BAD), (dict(Hk=3), BAD), (dict(Hk=-1), BAD), (dict(K=8), BAD),
    (dict(V=8), BAD), (dict(dtype=3), BAD), (dict(gate=2), BAD), (dict(lb=0.0), BAD), (dict(lb=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(n=1), BAD), (dict(n=0, slots=p()), BAD), (dict(q=0), BAD), (dict(st=0), BAD),
    (dict(K=144), UNSUP), (dict(V=256), UNSUP), (dict(K=40), UNSUP),
])
def test_decode_refusals(lib, kw, code):
    assert decode(lib, **kw) == code


def conv_prompt(lib, B=1, T=32, C=64, W=4, dtype=0, x=4096, xs=0, cu=None, host=None, n=0, h_in=0, y=4096, h_out=4096):
    return lib.kda_short_conv_prompt(B, T, C, W, dtype, p(x), xs, p(), None, cu, host, n, p(h_in), p(y), p(h_out), None)


def conv_step(lib, B=2, C=64, W=4, dtype=0, x=4096, xs=0, slots=None, n=2, h_in=4096, h_out=4096, y=4096):
    return lib.kda_short_conv_step(B, C, W, dtype, p(x), xs, p(), None, slots, n, p(h_in), p(h_out), p(y), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), BAD), (dict(C=0), BAD), (dict(W=0), BAD), (dict(dtype=9), BAD), (dict(x=0), BAD), (dict(y=0), BAD),
    (dict(xs=56), BAD), (dict(W=9), UNSUP), (dict(C=60), UNSUP), (dict(xs=68), UNSUP), (dict(x=4098), UNSUP),
    (dict(h_in=4104), UNSUP), (dict(h_out=4104), UNSUP),
])
def test_conv_refusals(lib, kw, code):
    assert conv_prompt(lib, **kw) == code
    assert conv_step(lib, **kw) == code


def test_conv_offsets_and_pools(lib):
    assert conv_prompt(lib, T=0) == BAD
    assert conv_prompt(lib, B=2, cu=p(), n=2) == BAD
    assert conv_prompt(lib, cu=p(), n=0) == BAD
    assert conv_prompt(lib, cu=p(), n=1, host=_lib.host_offsets([0, 31], 2)) == BAD
    assert conv_step(lib, n=1) == BAD
    assert conv_step(lib, h_in=0) == BAD


def pages(**kw):
    f = dict(layers=2, num_pages=64, num_seqs=8, max_pages=6, page_tokens=16, page_bytes=512, layer_stride=64 * 512)
    f.update(kw)
    return _lib.PagesDims(**f)


def fork(lib, d, n=1, pool=4096, req=4096, ok=4096, ws=4096, nb=1 << 20):
    return lib.kda_pages_fork(ctypes.byref(d), p(pool), p(), p(), p(), p(req), p(req), n, p(), p(), p(), p(ok), p(ws), nb,
                              None)


@pytest.mark.parametrize("kw,code", [
    (dict(layers=0), BAD), (dict(num_pages=0), BAD), (dict(num_seqs=0), BAD), (dict(max_pages=0), BAD),
    (dict(page_tokens=0), BAD), (dict(page_bytes=0), BAD), (dict(layer_stride=512), BAD),
    (dict(num_pages=(1 << 30) + 1, layers=1), UNSUP), (dict(num_seqs=1 << 20, max_pages=1 << 20), UNSUP),
    (dict(page_bytes=1 << 40, layers=1), UNSUP),
])
def test_pages_refusals(lib, kw, code):
    d = pages(**kw)
    assert fork(lib, d) == code
    assert lib.kda_pages_compact(ctypes.byref(d), p(), p(), p(), p(), p(), None, p(), 1 << 20, None) == code
    if not set(kw) & {"layers", "page_bytes", "layer_stride"}:
        assert lib.kda_pages_extend(ctypes.byref(d), *[p()] * 5, 1, *[p()] * 4, p(), 1 << 20, None) == code
        assert lib.kda_pages_free(ctypes.byref(d), *[p()] * 4, 1, *[p()] * 3, None) == code
        assert lib.kda_pages_workspace_size(ctypes.byref(d), 1) == 0


def test_pages_pointers_and_workspace(lib):
    d = pages()
    assert fork(lib, d, n=-1) == BAD
    assert fork(lib, d, pool=0) == BAD
    assert fork(lib, d, req=0) == BAD
    assert fork(lib, d, ok=0) == BAD
    need = lib.kda_pages_workspace_size(ctypes.byref(d), 1)
    assert need > 0
    assert fork(lib, d, nb=128) == WS
    assert fork(lib, d, ws=4096 + 4, nb=need) == WS
    copy = lambda **kw: lib.kda_pages_copy(*{**dict(layers=2, pb=64, dst=p(), ds=64 * 9, dn=9, src=p(), ss=64 * 9, sn=9,  # noqa: E731
                                                   a=p(), b=p(), n=1, st=None), **kw}.values())
    assert copy(layers=0) == BAD
    assert copy(pb=0) == BAD
    assert copy(ds=64) == BAD
    assert copy(dst=None) == BAD
    assert copy(a=None) == BAD
    assert copy(n=-1) == BAD


def test_binding_refuses_host_tensors():
    t = torch.zeros(2, 3, 4, 8)
    v = torch.zeros(4)
    with pytest.raises(ValueError):
        kda.ssm_scan(t, t[..., 0], t, t, v, v)
    with pytest.raises(ValueError):
        kda.pages_free(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_token_strides():
    stride = _lib._native().token_stride
    wide = torch.zeros(3, 5, 40)
    assert stride(wide[..., 8:32].unflatten(-1, (3, 8)), 2) == 40
    assert stride(wide[:, 0, :16], 1) == 200
    assert stride(torch.zeros(1, 1, 4, 8), 2) == 32
    with pytest.raises(ValueError):
        stride(wide[..., ::2], 2)                       # values not contiguous
    with pytest.raises(ValueError):
        stride(wide[:, :4], 2)                          # rows not evenly spaced


def test_binding_refuses_what_is_no_tensor():
    t, v = torch.zeros(2, 4, 8), torch.zeros(4)
    with pytest.raises(TypeError):
        kda.ssm_step([[0.0]], t[..., 0], t, t, v, v, state=torch.zeros(2, 4, 8, 8))
    with pytest.raises(TypeError):
        kda.pages_free(None, None, None, None)
    with pytest.raises(ValueError):
        kda.decode_step(t, t, t, t, t[..., 0], v, v, scale=1.0, gate="no such gate", state=torch.zeros(2, 4, 8, 8))
    with pytest.raises(ValueError):
        kda.short_conv_step(torch.zeros(2, 8), torch.zeros(8, 4), history=torch.zeros(2, 3, 8))
    with pytest.raises(TypeError):
        _lib._native().ssm_step(t)                      # too few arguments
