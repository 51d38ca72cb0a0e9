"""GPU parity of the gated linear recurrence against plain 64-bit references.

Tolerances, derived before the first run (u = 2^-24, half a step of fp32):
  * states and fp32 y: a factor a_t has a relative error of some 4 u (the sigmoid's exponential and reciprocal, the series,
    the rounding of 1 - e), and so has every input; they act over the memory of a state, up to a thousand tokens here, with
    mixed signs: 4 u sqrt(1000) = 7.5e-6 of the largest state, and 3e-5 with a margin for the largest of many;
  * bf16 y: 2^-8 |y| of storage, and 2e-3 of the rms for the same;
  * gradients: products of two such factors and gates, 1e-4 of the largest; da_log against the sum of its terms' sizes;
  * a step: a dozen roundings, 1e-5."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixer_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_delta_rule_sm_gb300 as kda  # noqa: E402
from gated_delta_rule_sm_gb300 import _lib  # noqa: E402
from kda_cases import rel_err  # noqa: E402

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SCAN, GRAD, STEP = 3e-5, 1e-4, 1e-5


def act_tol(dtype):
    return 2e-3 if dtype == "bf16" else SCAN


def inputs(seed, lead, C, dtype, strided=False, shift=0):
    """x and the gates, together slices of one projection where `strided`; shift: elements its base is off."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(*lead, 3 * C, generator=g).to(DT[dtype])
    if shift:
        flat = torch.zeros(z.numel() + shift, dtype=z.dtype, device=DEV)
        flat[shift:] = z.reshape(-1).to(DEV)
        z = flat[shift:].view(z.shape)
    x, gr, ir = z.to(DEV).chunk(3, dim=-1)
    if not strided and not shift:
        x, gr, ir = x.contiguous(), gr.contiguous(), ir.contiguous()
    a_log = torch.log(-torch.log(0.9 + 0.099 * torch.rand(C, generator=g))).to(DEV)
    return dict(x=x, g_raw=gr, i_raw=ir, a_log=a_log), g


def run(i, **kw):
    out = kda.gated_scan(i["x"], i["g_raw"], i["i_raw"], i["a_log"], **kw)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    return out


def flat(i):
    C = i["x"].shape[-1]
    return [ref.d(i[n]).reshape(-1, C) for n in ("x", "g_raw", "i_raw")] + [ref.d(i["a_log"])]


def check(i, offsets, s0, y, last, dtype):
    ry, rl = ref.gated(*flat(i), offsets, None if s0 is None else ref.d(s0))
    assert rel_err(y.reshape(ry.shape), ry.numpy(), dtype) <= act_tol(dtype)
    if last is not None:
        assert rel_err(last, rl.numpy(), "fp32") <= SCAN


# rows around a thread's, a record's and a tile's tokens, and tiles that hold several rows; channels around 32 and 64
@pytest.mark.parametrize("B,T,C,dtype,init", [
    (1, 1, 1, "bf16", True), (1, 1, 64, "fp32", False), (3, 1, 70, "bf16", True), (200, 1, 8, "bf16", True), (1, 15, 66, "bf16", True),
    (1, 16, 64, "bf16", False), (2, 17, 33, "fp32", True), (1, 64, 65, "bf16", True), (2, 127, 64, "bf16", True), (1, 128, 130, "fp32", True),
    (3, 129, 62, "bf16", True), (1, 300, 31, "bf16", False), (5, 40, 512, "bf16", True), (1, 1000, 100, "fp32", True), (2, 700, 96, "bf16", True),
])
def test_rows(B, T, C, dtype, init):
    i, g = inputs(B * T + C, (B, T), C, dtype)
    s0 = torch.randn(B, C, generator=g).to(DEV) if init else None
    y, last = run(i, initial_state=s0, output_final_state=True)
    check(i, [n * T for n in range(B + 1)], s0, y, last, dtype)
    y2, none = run(i, initial_state=s0)
    assert none is None and torch.equal(y, y2)


DOCS = [[5], [0, 3, 0, 0, 200, 128, 1, 64, 0], [127, 129, 256, 1, 1], [700, 0, 3, 650], [1] * 300, [0, 0, 40]]


@pytest.mark.parametrize("lengths", DOCS, ids=lambda n: str(n)[:24])
@pytest.mark.parametrize("C,dtype,init", [(64, "bf16", True), (70, "bf16", False), (35, "fp32", True)])
def test_documents(lengths, C, dtype, init):
    T, rows = sum(lengths), len(lengths)
    i, g = inputs(T + rows, (1, T), C, dtype, strided=True)
    s0 = torch.randn(rows, C, generator=g).to(DEV) if init else None
    off = [0, *np.cumsum(lengths).tolist()]
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    y, last = run(i, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    check(i, off, s0, y, last, dtype)
    y2, last2 = run(i, initial_state=s0, output_final_state=True, cu_seqlens=cu, cu_seqlens_host=off)
    assert torch.equal(y, y2) and torch.equal(last, last2)


def test_a_long_row_is_one_chain():
    """Hundreds of tiles: the look-back reaches past its 32 flags, and twice gives the same bits."""
    i, g = inputs(1, (1, 50021), 66, "bf16")
    s0 = torch.randn(1, 66, generator=g).to(DEV)
    y, last = run(i, initial_state=s0, output_final_state=True)
    for _ in range(3):
        y2, last2 = run(i, initial_state=s0, output_final_state=True)
        assert torch.equal(y, y2) and torch.equal(last, last2)
    x, gr, ir, al = flat(i)
    log_a = -torch.exp(al) * torch.sigmoid(gr)
    a, put = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(ir) * x
    h, want = ref.d(s0)[0], torch.empty_like(x)
    for t in range(x.shape[0]):
        h = a[t] * h + put[t]
        want[t] = h
    assert rel_err(y[0], want.numpy(), "bf16") <= act_tol("bf16")
    assert rel_err(last[0], h.numpy(), "fp32") <= SCAN


@pytest.mark.parametrize("C,dtype,shift", [(64, "bf16", 1), (64, "bf16", 2), (63, "bf16", 0), (40, "fp32", 1)])
def test_slices_at_any_element(C, dtype, shift):
    i, g = inputs(9, (2, 90), C, dtype, strided=True, shift=shift)
    y, last = run(i, output_final_state=True)
    check(i, [0, 90, 180], None, y, last, dtype)


def test_document_untouched_by_its_neighbours():
    lengths, off = [70, 150, 37], [0, 70, 220, 257]
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    i, g = inputs(7, (1, 257), 66, "bf16")
    s0 = torch.randn(3, 66, generator=g).to(DEV)
    y, last = run(i, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    j = {k: v.clone() for k, v in i.items()}
    for n in ("x", "g_raw", "i_raw"):
        j[n][:, :70] = float("nan")
        j[n][:, 220:] = float("inf")
    s1 = s0.clone()
    s1[0], s1[2] = float("nan"), float("inf")
    y2, last2 = run(j, initial_state=s1, output_final_state=True, cu_seqlens=cu)
    assert torch.equal(y[:, 70:220], y2[:, 70:220]) and torch.equal(last[1], last2[1])


@pytest.mark.parametrize("first", [5, 8, 30, 61, 64, 100])
def test_documents_beside_broken_ones_in_a_tile(first):
    """NaN in every input of the documents around it, at any place of a tile of tokens, forward and backward."""
    off = [0, first, first + 23, first + 60]
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    i, g = inputs(11, (1, off[-1]), 66, "bf16")
    s0, ds = torch.randn(3, 66, generator=g).to(DEV), torch.randn(3, 66, generator=g).to(DEV)
    dy = torch.randn(1, off[-1], 66, generator=g).to(DT["bf16"]).to(DEV)
    y, last = run(i, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    grads = kda.gated_scan_backward(i["x"], i["g_raw"], i["i_raw"], i["a_log"], dy, cu_seqlens=cu, initial_state=s0, dfinal_state=ds)
    mine = slice(off[1], off[2])
    j = {k: v.clone() for k, v in i.items()}
    others = [j["x"], j["g_raw"], j["i_raw"], dy]
    for t in others:
        t[:, :off[1]], t[:, off[2]:] = float("nan"), float("nan")
    for t in (s0, ds):
        t[0], t[2] = float("nan"), float("nan")
    y2, last2 = run(j, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    assert torch.equal(y[:, mine], y2[:, mine]) and torch.equal(last[1], last2[1])
    grads2 = kda.gated_scan_backward(j["x"], j["g_raw"], j["i_raw"], j["a_log"], dy, cu_seqlens=cu, initial_state=s0, dfinal_state=ds)
    for n in ("dx", "dg_raw", "di_raw"):
        assert torch.equal(grads[n][:, mine], grads2[n][:, mine]), n
    assert torch.equal(grads["dinitial_state"][1], grads2["dinitial_state"][1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_and_rates_at_their_ends(dtype):
    """Closed and open gates, rates from 0 to past fp32: no NaN, and the reference's values."""
    T, rates = 90, [-300.0, -60.0, -20.0, -1.4, -1.3, 0.0, 3.0, 88.0, 400.0]
    gates = [-300.0, -90.0, -41.0, -1.0, 0.0, 1.0, 41.0, 90.0, 300.0]
    C = len(rates) * len(gates)
    i, g = inputs(3, (1, T), C, dtype)
    i["a_log"] = torch.tensor(rates, device=DEV).repeat_interleave(len(gates)).contiguous()
    i["g_raw"] = torch.tensor(gates, device=DEV).repeat(len(rates)).expand(1, T, C).to(DT[dtype]).contiguous()
    i["i_raw"] = torch.tensor(gates, device=DEV).flip(0).repeat(len(rates)).expand(1, T, C).to(DT[dtype]).contiguous()
    s0 = torch.randn(1, C, generator=g).to(DEV)
    y, last = run(i, initial_state=s0, output_final_state=True)
    check(i, [0, T], s0, y, last, dtype)
    dy = torch.randn(1, T, C, generator=g).to(DT[dtype]).to(DEV)
    grads = kda.gated_scan_backward(i["x"], i["g_raw"], i["i_raw"], i["a_log"], dy, initial_state=s0)
    assert all(bool(torch.isfinite(t).all()) for t in grads.values())
    torch.cuda.synchronize()
    assert kda.device_status() == 0


def test_nan_and_infinity_stay_visible():
    """A NaN in any input of a token reaches its output and the later ones of its channel, and no other channel's."""
    for name in ("x", "g_raw", "i_raw"):
        i, _ = inputs(5, (1, 40), 64, "bf16")
        clean, _ = run(i)
        i[name][0, 11, 20] = float("nan")
        y, _ = run(i)
        assert bool(torch.isnan(y[0, 11:, 20]).all()), name
        y[0, 11:, 20] = clean[0, 11:, 20]
        assert torch.equal(y, clean)


# ------------------------------------------------------------------------------------------- gradients


def check_grads(i, offsets, s0, dy, dlast, grads):
    C = i["x"].shape[-1]
    want, terms = ref.gated_grads(*[i[n].reshape(-1, C) for n in ("x", "g_raw", "i_raw")], i["a_log"], offsets, s0, dy.reshape(-1, C), dlast)
    for n in ("dx", "dg_raw", "di_raw", "dinitial_state"):
        assert rel_err(grads[n].reshape(want[n].shape), want[n].numpy(), "fp32") <= GRAD, n
    assert bool(((ref.d(grads["da_log"]) - want["da_log"]).abs() <= GRAD * terms + 1e-30).all())


def backward(i, dy, **kw):
    g = kda.gated_scan_backward(i["x"], i["g_raw"], i["i_raw"], i["a_log"], dy, **kw)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    return g


@pytest.mark.parametrize("B,T,C,dtype,init", [
    (1, 1, 1, "bf16", True), (3, 1, 70, "bf16", True), (1, 7, 64, "bf16", False), (1, 8, 66, "bf16", True), (2, 9, 33, "fp32", True),
    (1, 63, 64, "bf16", True), (2, 64, 64, "bf16", True), (1, 65, 65, "bf16", True), (3, 129, 62, "bf16", True), (1, 300, 40, "fp32", True),
    (2, 333, 96, "bf16", False),
])
def test_gradients_of_rows(B, T, C, dtype, init):
    i, g = inputs(B * T + C, (B, T), C, dtype)
    s0 = torch.randn(B, C, generator=g).to(DEV) if init else None
    dlast = torch.randn(B, C, generator=g).to(DEV) if init else None
    dy = torch.randn(B, T, C, generator=g).to(DT[dtype]).to(DEV)
    grads = backward(i, dy, initial_state=s0, dfinal_state=dlast)
    check_grads(i, [n * T for n in range(B + 1)], s0, dy, dlast, grads)


@pytest.mark.parametrize("lengths", DOCS[:4] + [[1] * 90, [0, 0, 40]], ids=lambda n: str(n)[:24])
@pytest.mark.parametrize("C,dtype", [(64, "bf16"), (35, "fp32")])
def test_gradients_of_documents(lengths, C, dtype):
    T, rows = sum(lengths), len(lengths)
    i, g = inputs(T + rows, (1, T), C, dtype, strided=True)
    s0, dlast = torch.randn(rows, C, generator=g).to(DEV), torch.randn(rows, C, generator=g).to(DEV)
    off = [0, *np.cumsum(lengths).tolist()]
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    dy = torch.randn(1, T, C, generator=g).to(DT[dtype]).to(DEV)
    kw = dict(initial_state=s0, dfinal_state=dlast, cu_seqlens=cu)
    grads = backward(i, dy, **kw)
    check_grads(i, off, s0, dy, dlast, grads)
    # with the forward's record: the same bits; without the initial state's gradient: the others the same
    saved = torch.empty(kda.gated_scan_saved_size(i["x"]), dtype=torch.uint8, device=DEV)
    run(i, initial_state=s0, cu_seqlens=cu, saved=saved)
    again = backward(i, dy, saved=saved, want_dinitial_state=False, **kw)
    assert again["dinitial_state"] is None
    for n in ("dx", "dg_raw", "di_raw", "da_log"):
        assert torch.equal(again[n], grads[n]), n


def check_grads_at_the_ends(i, s0, dy, dlast):
    """Against the chain rule, every gradient by its own terms.  Derived before the first run, u = 2^-24: GRAD for the products, as above;
    a rate above 1/4 forms log a in exponents of up to |a_log| + |g|, three roundings of u each there, which the state and its
    gradient take over once more: 8 u (|a_log| + |g|); a decay is 1 - e, off by u whatever it is, twice, with a factor log a that matters
    down to e^-20: 2^-21 min(|log a|, 20); 1 - sigmoid and the input's sigmoid stop at 2^-60: 2^-59."""
    T, C = i["x"].shape[1:]
    grads = backward(i, dy, initial_state=s0, dfinal_state=dlast)
    want, z = ref.gated_back(*[i[n].reshape(-1, C) for n in ("x", "g_raw", "i_raw")], i["a_log"], [0, T], s0, dy.reshape(-1, C), dlast)
    rel = GRAD + 8 * 2.0 ** -24 * (ref.d(i["a_log"]).abs() + ref.d(i["g_raw"][0]).clamp(-400, 400).abs())
    stop = 2.0 ** -59 * z["M"] * (z["H"] + z["X"] + 1)
    tol = rel * z["terms"] + 2.0 ** -21 * z["log_a"].abs().clamp(max=20) * z["M"] * (z["H"] + z["U"]) + stop
    tols = dict(dx=rel * z["M"] * z["root"] * z["keep"] + stop, dg_raw=tol, di_raw=rel * z["M"] * z["root"] * z["U"] + stop, da_log=tol.sum(0),
                dinitial_state=rel.amax(0) * z["M"] + stop)
    for n, t in tols.items():
        err = (ref.d(grads[n]).reshape(want[n].shape) - want[n]).abs() / t
        assert float(err.max()) <= 1.0, (n, float(err.max()), int(err.amax(0).argmax()) if err.dim() > 1 else int(err.argmax()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_of_closed_gates(dtype):
    """Gates that a large negative logit closes, at rates that the ordinary tiles take: whole tiles and those of the row's ends."""
    T, rates = 256, [0.01, 0.05, 0.1, 0.24]
    gates = [-1.0, -20.0, -30.0, -40.0, -41.0, -42.0, -45.0, -50.0, -55.0, -60.0, -70.0, -80.0, -90.0, -300.0, -1e4, -np.inf]
    C = len(rates) * len(gates)
    i, g = inputs(13, (1, T), C, dtype)
    i["a_log"] = torch.log(torch.tensor(rates)).to(DEV).repeat_interleave(len(gates)).contiguous()
    i["g_raw"] = torch.tensor(gates, device=DEV).repeat(len(rates)).expand(1, T, C).to(DT[dtype]).contiguous()
    s0, dlast = (torch.randn(1, C, generator=g).to(DEV) for _ in range(2))
    check_grads_at_the_ends(i, s0, torch.randn(1, T, C, generator=g).to(DT[dtype]).to(DEV), dlast)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_of_gates_and_rates_at_their_ends(dtype):
    T, rates = 90, [-300.0, -60.0, -20.0, -1.4, -1.3, 0.0, 3.0, 88.0, 400.0]
    gates = [-300.0, -90.0, -60.0, -41.0, -1.0, 0.0, 1.0, 41.0, 90.0, 300.0]
    C = len(rates) * len(gates)
    i, g = inputs(3, (1, T), C, dtype)
    i["a_log"] = torch.tensor(rates, device=DEV).repeat_interleave(len(gates)).contiguous()
    i["g_raw"] = torch.tensor(gates, device=DEV).repeat(len(rates)).expand(1, T, C).to(DT[dtype]).contiguous()
    i["i_raw"] = torch.tensor(gates, device=DEV).flip(0).repeat(len(rates)).expand(1, T, C).to(DT[dtype]).contiguous()
    s0 = torch.randn(1, C, generator=g).to(DEV)
    check_grads_at_the_ends(i, s0, torch.randn(1, T, C, generator=g).to(DT[dtype]).to(DEV), None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_fast_rates_keep_their_small_decays(dtype):
    """Decays down to e^-50: states that only decay, and the gradients of their rates, by their own size.  With u = 2^-24: log a is off
    by 8 u (|a_log| + |g|) and 16 u of itself (as above), a decay by |log a| times that and 2^-21 of itself (one exponential whose
    argument has been rounded); a gradient's term takes it twice more, with GRAD for the other factors."""
    B, T, rates = 40, 3, [0.3, 1.0, 4.0, 12.0, 30.0, 60.0, 100.0, 0.1]
    C = 9 * len(rates)
    i, g = inputs(17, (B, T), C, dtype)
    i["a_log"] = torch.log(torch.tensor(rates)).to(DEV).repeat_interleave(9).contiguous()
    s0, dlast = (torch.randn(B, C, generator=g).to(DEV) for _ in range(2))
    al, gr = ref.d(i["a_log"]), ref.d(i["g_raw"])
    log_a = -torch.exp(al) * torch.sigmoid(gr)
    off = log_a.abs() * 2.0 ** -24 * (8 * (al.abs() + gr.abs()) + 16) + 2.0 ** -21          # of each decay, relative
    # closed input gates: what is left of the state is the product of the decays
    only = dict(i, x=torch.zeros_like(i["x"]))
    y, last = run(only, initial_state=s0, output_final_state=True)
    want, tol = torch.exp(log_a.cumsum(1)) * ref.d(s0)[:, None], off.cumsum(1) + (2.0 ** -8 if dtype == "bf16" else 0.0)
    assert bool(((ref.d(y) - want).abs() <= tol * want.abs() + 1e-37).all())
    assert bool(((ref.d(last) - want[:, -1]).abs() <= off.sum(1) * want[:, -1].abs() + 1e-37).all())
    step = {n: t[:, 0].contiguous() if t.dim() == 3 else t for n, t in only.items()}
    y, pool = kda.gated_step(step["x"], step["g_raw"], step["i_raw"], step["a_log"], state=s0.clone())
    assert bool(((ref.d(pool) - want[:, 0]).abs() <= off[:, 0] * want[:, 0].abs() + 1e-37).all())
    # the gradients of the rates, by the sizes of their terms
    dy = torch.randn(B, T, C, generator=g).to(DT[dtype]).to(DEV)
    grads = backward(i, dy, initial_state=s0, dfinal_state=dlast)
    want, terms = ref.gated_grads(*[i[n].reshape(-1, C) for n in ("x", "g_raw", "i_raw")], i["a_log"], [n * T for n in range(B + 1)], s0,
                                  dy.reshape(-1, C), dlast)
    rel = GRAD + 3 * off.reshape(-1, C).amax(0)
    assert bool(((ref.d(grads["da_log"]) - want["da_log"]).abs() <= rel * terms + 1e-36).all())


def test_gradients_against_differences():
    """Along a direction, the gradients' product is the slope of the 64-bit forward (central differences, whose own error
    is h^2 of the third derivative, about 1e-8 here)."""
    i, g = inputs(11, (1, 150), 40, "fp32")
    off, s0 = [0, 60, 150], torch.randn(2, 40, generator=g)
    dy, dlast = torch.randn(150, 40, generator=g), torch.randn(2, 40, generator=g)
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    grads = backward(i, dy.to(DEV)[None], cu_seqlens=cu, initial_state=s0.to(DEV), dfinal_state=dlast.to(DEV))
    at = flat(i) + [s0.double()]
    names = ("dx", "dg_raw", "di_raw", "da_log", "dinitial_state")
    for k, n in enumerate(names):
        v = torch.randn(at[k].shape, generator=g).double()

        def value(h):
            z = [t + h * v if j == k else t for j, t in enumerate(at)]
            y, last = ref.gated(*z[:4], off, z[4])
            return float((y * dy.double()).sum() + (last * dlast.double()).sum())

        slope = (value(1e-4) - value(-1e-4)) / 2e-4
        mine = float((ref.d(grads[n]).reshape(v.shape) * v).sum())
        size = float((ref.d(grads[n]).reshape(v.shape) * v).abs().sum())
        assert abs(slope - mine) <= 1e-5 * size, (n, slope, mine)


def test_long_gradients_are_one_chain():
    i, g = inputs(21, (1, 20011), 64, "bf16")
    dy = torch.randn(1, 20011, 64, generator=g).bfloat16().to(DEV)
    first = backward(i, dy)
    again = backward(i, dy)
    assert all(torch.equal(first[n], again[n]) for n in first)
    x, gr, ir, al = flat(i)
    log_a = -torch.exp(al) * torch.sigmoid(gr)
    a, root = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    back, dx = torch.zeros(64, dtype=torch.float64), torch.empty_like(x)
    for t in range(x.shape[0] - 1, -1, -1):
        lam = ref.d(dy[0, t]) + back
        dx[t] = lam * root[t] * torch.sigmoid(ir[t])
        back = a[t] * lam
    assert rel_err(first["dx"][0], dx.numpy(), "fp32") <= GRAD
    assert rel_err(first["dinitial_state"][0], back.numpy(), "fp32") <= GRAD


# ------------------------------------------------------------------------------------------- step


@pytest.mark.parametrize("B,C,dtype", [(1, 1, "bf16"), (1, 4096, "bf16"), (9, 70, "bf16"), (33, 257, "fp32"), (128, 515, "bf16")])
def test_step(B, C, dtype):
    i, g = inputs(B + C, (B,), C, dtype, strided=True)
    pool = torch.randn(B + 5, C, generator=g).to(DEV)
    slots = torch.randperm(B + 5, generator=g)[:B].to(torch.int32)
    if B > 3:
        slots[2] = -1
    new = torch.full_like(pool, 7.0)
    y, got = kda.gated_step(i["x"], i["g_raw"], i["i_raw"], i["a_log"], state=pool, slots=slots.to(DEV), state_out=new)
    assert got is new
    live = [r for r in range(B) if slots[r] >= 0]
    x, gr, ir, al = flat(i)
    want_y, want = torch.zeros_like(x), ref.d(new).clone().fill_(7.0)
    for r in live:
        h = ref.gated(x[r:r + 1], gr[r:r + 1], ir[r:r + 1], al, [0, 1], ref.d(pool[slots[r]])[None])[1][0]
        want_y[r] = want[slots[r]] = h
    assert rel_err(y, want_y.numpy(), dtype) <= (2e-3 if dtype == "bf16" else STEP)
    assert rel_err(new, want.numpy(), "fp32") <= STEP
    y2, same = kda.gated_step(i["x"], i["g_raw"], i["i_raw"], i["a_log"], state=pool, slots=slots.to(DEV))
    assert same is pool and torch.equal(y, y2)
    for r in live:
        assert torch.equal(pool[slots[r]], new[slots[r]])


def test_steps_continue_a_scan():
    """The scan's state and steps from it: the same outputs as the scan over all tokens, to fp32 rounding."""
    i, _ = inputs(2, (3, 80), 64, "fp32")
    whole, _ = run(i)
    cut = {n: (t[:, :73].contiguous() if t.dim() == 3 else t) for n, t in i.items()}
    _, pool = run(cut, output_final_state=True)
    for t in range(73, 80):
        y, pool = kda.gated_step(*[i[n][:, t] for n in ("x", "g_raw", "i_raw")], i["a_log"], state=pool)
        assert float((y - whole[:, t]).abs().max()) <= STEP * float(whole.abs().max())


def test_step_slot_past_the_pool_is_an_idle_row():
    i, g = inputs(2, (2,), 64, "bf16")
    pool = torch.randn(3, 64, generator=g).to(DEV)
    kept = pool.clone()
    y, _ = kda.gated_step(i["x"], i["g_raw"], i["i_raw"], i["a_log"], state=pool, slots=torch.tensor([3, -1], dtype=torch.int32, device=DEV))
    assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG
    assert torch.equal(pool, kept) and not bool(y.any())


# ------------------------------------------------------------------------------------------- calls


def test_in_place():
    i, g = inputs(4, (1, 400), 66, "bf16")
    cu = torch.tensor([0, 100, 100, 400], dtype=torch.int32, device=DEV)
    s0 = torch.randn(3, 66, generator=g).to(DEV)
    y, last = run(i, initial_state=s0, output_final_state=True, cu_seqlens=cu)
    x, s = i["x"].clone(), s0.clone()
    y2, last2 = kda.gated_scan(x, i["g_raw"], i["i_raw"], i["a_log"], cu_seqlens=cu, initial_state=s, output_final_state=True, out=x, final_state=s)
    assert y2 is x and last2 is s and torch.equal(x, y) and torch.equal(s, last)


def test_offsets_that_break_the_contract():
    i, g = inputs(4, (1, 300), 64, "bf16")
    s0 = torch.randn(2, 64, generator=g).to(DEV)
    for bad in ([0, 200, 299], [1, 200, 300], [0, 301, 300]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        out = torch.full_like(i["x"], 3.0)
        _, last = kda.gated_scan(i["x"], i["g_raw"], i["i_raw"], i["a_log"], cu_seqlens=cu, initial_state=s0, output_final_state=True, out=out)
        assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG
        assert bool((out == 3.0).all()) and torch.equal(last, s0)
        grads = kda.gated_scan_backward(i["x"], i["g_raw"], i["i_raw"], i["a_log"], i["x"], cu_seqlens=cu, initial_state=s0, dfinal_state=s0)
        assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG
        assert torch.equal(grads["dinitial_state"], s0) and not bool(grads["da_log"].any())
        with pytest.raises(kda.KdaError):
            kda.gated_scan(i["x"], i["g_raw"], i["i_raw"], i["a_log"], cu_seqlens=cu, cu_seqlens_host=bad)


def test_streams_and_captured_graphs():
    """Two streams at once, and two graphs captured on one stream, replayed in turn and together with eager calls."""
    sets = [inputs(s, (1, 2000), 128, "bf16")[0] for s in (1, 2)]
    want = [run(i, output_final_state=True) for i in sets]
    dys = [torch.randn_like(i["x"]) for i in sets]
    grads = [backward(i, dy) for i, dy in zip(sets, dys)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for k in range(6):
        i, st = sets[k % 2], streams[k % 2]
        got.append(kda.gated_scan(i["x"], i["g_raw"], i["i_raw"], i["a_log"], output_final_state=True, stream=st))
    torch.cuda.synchronize()
    for k, (y, last) in enumerate(got):
        assert torch.equal(y, want[k % 2][0]) and torch.equal(last, want[k % 2][1])
    graphs, outs = [], []
    for i, dy in zip(sets, dys):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, last = kda.gated_scan(i["x"], i["g_raw"], i["i_raw"], i["a_log"], output_final_state=True)
            gr = kda.gated_scan_backward(i["x"], i["g_raw"], i["i_raw"], i["a_log"], dy)
        graphs.append(graph)
        outs.append((y, last, gr))
    for k in (0, 1, 0):
        graphs[k].replay()
        with torch.cuda.stream(streams[0]):
            graphs[1 - k].replay()
        other = run(sets[1], output_final_state=True)
        torch.cuda.synchronize()
        assert torch.equal(other[0], want[1][0])
        for (y, last, gr), (wy, wl), wg in zip(outs, want, grads):
            assert torch.equal(y, wy) and torch.equal(last, wl)
            assert all(torch.equal(gr[n], wg[n]) for n in wg)
        for y, _, _ in outs:
            y.fill_(9.0)


@pytest.mark.parametrize("what", ["shape", "dtype", "rate", "state", "expanded", "saved", "overlap", "gate", "dy"])
def test_refusals(what):
    i, _ = inputs(1, (2, 20), 64, "bf16")
    a, kw = [i["x"], i["g_raw"], i["i_raw"], i["a_log"]], {}
    err = ValueError
    if what == "shape":
        a[1] = a[1][:, :19]
    elif what == "dtype":
        a[2] = a[2].float()
    elif what == "rate":
        a[3] = a[3][:63].contiguous()
    elif what == "state":
        kw["initial_state"] = torch.zeros(3, 64, device=DEV)
    elif what == "expanded":
        a[0] = a[0][:, :1].expand(2, 20, 64)
    elif what == "saved":
        kw["saved"], err = torch.empty(16, dtype=torch.uint8, device=DEV), kda.KdaError
    elif what == "overlap":
        kw["out"], err = i["g_raw"], kda.KdaError
    elif what == "gate":
        a[1] = a[1].cpu()
    else:
        with pytest.raises(ValueError):
            kda.gated_scan_backward(*a, i["x"].float())
        return
    with pytest.raises(err):
        kda.gated_scan(*a, **kw)
