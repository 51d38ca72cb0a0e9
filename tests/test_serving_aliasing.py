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
