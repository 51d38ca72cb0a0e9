"""Calls whose results would lie over what other blocks of the same launch still read: refused on the host."""
from __future__ import annotations

import ctypes

import pytest

import __graft_entry__
from gated_delta_rule_sm_gb300 import _lib

BAD = _lib.KDA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


def p(addr):
    return ctypes.c_void_p(addr) if addr else None


X, Y, H0, H1 = 1 << 20, 2 << 20, 3 << 20, 4 << 20
T, C, W = 32, 64, 4           # bf16: x and y 4096 bytes each, a history 384


# (no call here is valid: one that passed the checks would be launched on these addresses)
@pytest.mark.parametrize("kw", [
    dict(y=X), dict(y=X + 4096 - 16), dict(y=X - 4096 + 16), dict(y=X + 6 * 4096, xs=512),     # y and x, x strided
    dict(y=H0), dict(y=H0 - 4096 + 16), dict(y=H1 + 384 - 16),                                 # y and the histories
    dict(h1=X), dict(h1=X + 4096 - 16), dict(h1=H0 + 16), dict(h1=H0 - 384 + 16),              # the final history
])
def test_conv_prompt_results_over_its_inputs(lib, kw):
    a = dict(x=X, y=Y, h0=H0, h1=H1, xs=0)
    a.update(kw)
    assert lib.kda_short_conv_prompt(1, T, C, W, _lib.KDA_BF16, p(a["x"]), a["xs"], p(64), None, None, None, 0, p(a["h0"]),
                                     p(a["y"]), p(a["h1"]), None) == BAD


@pytest.mark.parametrize("kw", [
    dict(y="x", xs=272), dict(y="x", dy=16), dict(y="x", dy=-16), dict(y="b"), dict(y="c"), dict(y="c", dy=-16), dict(y="dt"),
    dict(y="S0"), dict(y="ST"), dict(ST="x"), dict(ST="b"), dict(ST="c"), dict(ST="dt"), dict(ST="S0", dST=16),
])
def test_scan_results_over_its_inputs(lib, kw):
    at = dict(x=1 << 24, dt=2 << 24, b=3 << 24, c=4 << 24, S0=5 << 24, ST=6 << 24, y=7 << 24)
    for out in ("y", "ST"):
        if out in kw:
            at[out] = at[kw[out]] + kw.get("d" + out, 0)
    dims = _lib.SsmDims(1, 100, 4, 2, 64, 64, _lib.KDA_BF16, 0, kw.get("xs", 0), 0, 0, 0)
    size = lib.kda_ssm_fwd_workspace_size(ctypes.byref(dims))
    got = lib.kda_ssm_fwd(ctypes.byref(dims), p(at["x"]), p(at["dt"]), p(at["b"]), p(at["c"]), p(64), p(64), None, None, None,
                          p(at["S0"]), p(at["y"]), p(at["ST"]), p(8 << 24), size, None)
    assert got == BAD
