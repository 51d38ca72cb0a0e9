"""GPU parity of the serving operators against plain 64-bit references.

Tolerances, per kind of result (errors over the largest reference magnitude unless stated):
  * states of single steps and fp32 outputs: a dozen fp32 roundings of 2^-24 each on exact inputs, 1e-5;
  * states of a scan: products of up to some hundred factors exp(D a), each with a relative error of a few
    2^-24, and on the tensor cores one operand kept as two bf16 values (2^-17): 3e-5;
  * bf16 results, after the storage rounding 2^-8 |r| is allowed, over the rms: 2e-3 where the arithmetic is
    fp32, and 2e-2 (the package's bf16 tolerance) where products round one operand to bf16.
Whole numbers and copied pages are equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_delta_rule_sm_gb300 as kda  # noqa: E402
from kda_cases import rel_err  # noqa: E402

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
STEP, SCAN = 1e-5, 3e-5


def act_tol(dtype, rounded):
    return (2e-2 if rounded else 2e-3) if dtype == "bf16" else SCAN


def randn(gen, *shape):
    return torch.randn(shape, generator=gen)


def ssm_inputs(seed, lead, H, G, N, P, dtype, strided=False, shift=0):
    """lead: the token axes.  strided: x, b, c as slices of one projection; shift: elements its base is off."""
    g = torch.Generator().manual_seed(seed)
    widths = [H * P, G * N, G * N]
    xbc = randn(g, *lead, sum(widths)).to(DT[dtype])
    if shift:
        flat = torch.zeros(xbc.numel() + shift, dtype=xbc.dtype, device=DEV)
        flat[shift:] = xbc.reshape(-1).to(DEV)
        xbc = flat[shift:].view(xbc.shape)
    xbc = xbc.to(DEV)
    x, b, c = xbc.split(widths, dim=-1)
    if not strided and not shift:
        x, b, c = x.contiguous(), b.contiguous(), c.contiguous()
    dt = (0.5 * randn(g, *lead, H)).to(DT[dtype]).to(DEV)
    step = torch.exp(np.log(1e-3) + torch.rand(H, generator=g) * np.log(1e2))
    return dict(x=x.unflatten(-1, (H, P)), dt_raw=dt, b=b.unflatten(-1, (G, N)), c=c.unflatten(-1, (G, N)),
                a_log=torch.log(1 + 15 * torch.rand(H, generator=g)).to(DEV),
                dt_bias=(step + torch.log(-torch.expm1(-step))).to(DEV),
                d_skip=(1 + 0.1 * randn(g, H)).to(DEV)), g


def check_scan(i, offsets, S0, y, S, dtype, rounded):
    B, T, H, P = i["x"].shape
    flat = [i[n].reshape(B * T, *i[n].shape[2:]) for n in ("x", "dt_raw", "b", "c")]
    ry, rS = ref.ssm(*flat, i["a_log"], i["dt_bias"], i["d_skip"], offsets, S0)
    assert rel_err(y.reshape(B * T, H, P), ry.numpy(), dtype) <= act_tol(dtype, rounded)
    if S is not None:
        assert rel_err(S, rS.numpy(), "fp32") <= SCAN


ARGS = ("x", "dt_raw", "b", "c", "a_log", "dt_bias", "d_skip")


def run_scan(i, **kw):
    out = kda.ssm_scan(*[i[n] for n in ARGS], **kw)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    return out


# rows of one token, around a chunk's end, several chunks; heads to a group odd and even; N, P at and off
# the sizes the tensor-core tiles have
@pytest.mark.parametrize("B,T,H,G,N,P,dtype,init", [
    (1, 1, 2, 1, 64, 64, "bf16", True), (2, 1, 3, 3, 16, 16, "bf16", False), (1, 127, 4, 2, 64, 64, "bf16", False),
    (1, 128, 2, 1, 128, 64, "bf16", True), (2, 129, 4, 1, 128, 128, "bf16", True), (1, 300, 6, 2, 128, 64, "bf16", True),
    (1, 257, 3, 1, 96, 80, "bf16", True), (2, 200, 5, 1, 48, 40, "bf16", True), (1, 130, 2, 2, 24, 8, "bf16", False),
    (1, 140, 4, 2, 256, 64, "bf16", True), (1, 70, 2, 1, 64, 256, "bf16", True), (1, 90, 2, 1, 20, 12, "bf16", True),
    (1, 1, 1, 1, 1, 1, "fp32", True), (2, 150, 6, 2, 48, 40, "fp32", True), (1, 200, 4, 4, 128, 64, "fp32", False),
    (1, 40, 2, 1, 250, 33, "fp32", True), (1, 1300, 2, 1, 64, 64, "bf16", True), (1, 1300, 2, 1, 32, 32, "fp32", True),
])
def test_scan_rows(B, T, H, G, N, P, dtype, init):
    i, g = ssm_inputs(B * T + N + P, (B, T), H, G, N, P, dtype)
    S0 = randn(g, B, H, N, P).to(DEV) if init else None
    y, S = run_scan(i, initial_state=S0, output_final_state=True)
    check_scan(i, [n * T for n in range(B + 1)], S0, y, S, dtype, dtype == "bf16")


@pytest.mark.parametrize("lengths", [[5], [0, 3, 0, 0, 200, 128, 1, 64, 0], [127, 129, 256, 1, 1], [700, 0, 3, 650]])
@pytest.mark.parametrize("dtype,init", [("bf16", True), ("bf16", False), ("fp32", True)])
def test_scan_documents(lengths, dtype, init):
    T, rows = sum(lengths), len(lengths)
    i, g = ssm_inputs(T + rows, (1, T), 4, 2, 64, 64, dtype)
    S0 = randn(g, rows, 4, 64, 64).to(DEV) if init else None
    off = [0, *np.cumsum(lengths).tolist()]
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True, cu_seqlens=cu)
    check_scan(i, off, S0, y, S, dtype, dtype == "bf16")
    y2, S2 = run_scan(i, initial_state=S0, output_final_state=True, cu_seqlens=cu, cu_seqlens_host=off)
    assert torch.equal(y, y2) and torch.equal(S, S2)


@pytest.mark.parametrize("H,G,N,P", [(4, 2, 64, 64), (3, 1, 128, 64), (2, 1, 128, 128), (2, 2, 256, 96)])
def test_scan_document_untouched_by_its_neighbours(H, G, N, P):
    """NaN and infinities in the documents around one, and in its neighbours' states, leave it as it was."""
    lengths = [70, 150, 37]
    off = [0, 70, 220, 257]
    i, g = ssm_inputs(7, (1, 257), H, G, N, P, "bf16")
    S0 = randn(g, 3, H, N, P).to(DEV)
    cu = torch.tensor(off, dtype=torch.int32, device=DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True, cu_seqlens=cu)
    j = {k: v.clone() for k, v in i.items()}
    for n in ("x", "b", "c", "dt_raw"):
        j[n][:, :70] = float("nan")
        j[n][:, 220:] = float("inf")
    S1 = S0.clone()
    S1[0], S1[2] = float("inf"), float("nan")
    y1, S_1 = run_scan(j, initial_state=S1, output_final_state=True, cu_seqlens=cu)
    assert len(lengths) == 3
    assert torch.equal(y[:, 70:220], y1[:, 70:220]) and torch.equal(S[1], S_1[1])


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype,N,P", [("bf16", 64, 64), ("bf16", 20, 36), ("fp32", 48, 40)])
def test_scan_reads_slices_of_a_projection(dtype, N, P, shift):
    """x, b and c as slices; a base off the 16-byte boundary included.  The values are the contiguous call's."""
    i, g = ssm_inputs(3, (2, 150), 4, 2, N, P, dtype, strided=True, shift=shift)
    S0 = randn(g, 2, 4, N, P).to(DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True)
    check_scan(i, [0, 150, 300], S0, y, S, dtype, dtype == "bf16")
    k = {n: t.contiguous().clone() for n, t in i.items()}
    y2, S2 = run_scan(k, initial_state=S0, output_final_state=True)
    assert rel_err(y, ref.d(y2).numpy(), dtype) <= act_tol(dtype, True)
    assert rel_err(S, ref.d(S2).numpy(), "fp32") <= SCAN


def test_scan_without_skip_and_state():
    i, _ = ssm_inputs(11, (1, 200), 4, 1, 64, 64, "bf16")
    i["d_skip"] = None
    y, S = run_scan(i)
    assert S is None
    check_scan(i, [0, 200], None, y, None, "bf16", True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_strong_and_weak_decay(dtype):
    """Steps so large that a token forgets everything (the decay underflows), and so small that nothing fades."""
    i, g = ssm_inputs(13, (1, 300), 4, 2, 64, 64, dtype)
    i["dt_raw"][:, :, 0] = 40.0     # exp(-D e^a_log) is 0
    i["dt_raw"][:, 100:104, 1] = 60.0
    i["dt_raw"][:, :, 2] = -30.0    # D about 1e-13
    S0 = randn(g, 1, 4, 64, 64).to(DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True)
    flat = [i[n][0] for n in ("x", "dt_raw", "b", "c")]
    ry, rS = ref.ssm(*flat, i["a_log"], i["dt_bias"], i["d_skip"], [0, 300], S0)
    for h in range(4):              # heads differ by orders of magnitude
        assert rel_err(y[0, :, h], ry[:, h].numpy(), dtype) <= act_tol(dtype, True), h
        assert rel_err(S[0, h], rS[0, h].numpy(), "fp32") <= SCAN, h


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_in_two_calls(dtype):
    """A prompt in two calls through the carried state is the prompt in one."""
    i, _ = ssm_inputs(17, (1, 421), 4, 2, 64, 64, dtype)
    y, S = run_scan(i, output_final_state=True)
    cut = {n: (i[n][:, :201].contiguous() if n in ("x", "b", "c", "dt_raw") else i[n]) for n in i}
    rest = {n: (i[n][:, 201:].contiguous() if n in ("x", "b", "c", "dt_raw") else i[n]) for n in i}
    y1, S1 = run_scan(cut, output_final_state=True)
    y2, S2 = run_scan(rest, initial_state=S1, output_final_state=True)
    assert rel_err(torch.cat([y1, y2], 1), ref.d(y).numpy(), dtype) <= act_tol(dtype, True)
    assert rel_err(S2, ref.d(S).numpy(), "fp32") <= 2 * SCAN


@pytest.mark.parametrize("offsets", [[0, 150, 100, 300], [5, 100, 200, 300], [0, 100, 200, 290]])
def test_scan_bad_device_offsets_are_reported(offsets):
    i, g = ssm_inputs(19, (1, 300), 4, 2, 64, 64, "bf16")
    S0 = randn(g, 3, 4, 64, 64).to(DEV)
    out = torch.full_like(i["x"], float("nan"))
    cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    _, S = kda.ssm_scan(*[i[n] for n in ARGS], cu_seqlens=cu, initial_state=S0, output_final_state=True, out=out)
    hist = torch.full((3, 3, 64), float("nan"), device=DEV, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert kda.device_status() == 1
    assert bool(torch.isnan(out.float()).all()) and torch.equal(S, S0)
    x = i["x"][:, :, 0].contiguous()
    co = torch.full_like(x, float("nan"))
    kda.short_conv_prompt(x, torch.zeros(64, 4, device=DEV), cu_seqlens=cu, out=co, final_history=hist)
    torch.cuda.synchronize()
    assert kda.device_status() == 1
    assert bool(torch.isnan(co.float()).all()) and bool(torch.isnan(hist.float()).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("init", [True, False])
def test_scan_of_long_documents_in_segments(dtype, init):
    """Documents of many segments, of a segment and a token, and of none, side by side."""
    lengths = [2600, 0, 5, 1024, 129, 2817, 1, 513]
    off = [0, *np.cumsum(lengths).tolist()]
    i, g = ssm_inputs(37, (1, off[-1]), 4, 2, 64, 16, dtype)
    S0 = randn(g, len(lengths), 4, 64, 16).to(DEV) if init else None
    y, S = run_scan(i, initial_state=S0, output_final_state=True, cu_seqlens=torch.tensor(off, dtype=torch.int32, device=DEV))
    check_scan(i, off, S0, y, S, dtype, dtype == "bf16")


def test_scan_of_many_chunks_to_a_segment():
    """Enough heads and tokens that a segment is longer than any ring of buffers.  With so many values the bound of
    y is taken for each: its storage rounding, and one rounding to bf16 (2^-9, doubled for the fp32 sums) of each
    token's factor inside a chunk of 128."""
    T, H, N, P, Q = 16300, 32, 128, 8, 128
    i, g = ssm_inputs(41, (1, T), H, 1, N, P, "bf16")
    S0 = randn(g, 1, H, N, P).to(DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True)
    x, dt, b, c = (ref.d(i[n][0]) for n in ("x", "dt_raw", "b", "c"))
    ry, rS = ref.ssm(x, dt, b, c, i["a_log"], i["dt_bias"], i["d_skip"], [0, T], S0)
    delta = ref.softplus(dt + ref.d(i["dt_bias"]))
    la = -torch.exp(ref.d(i["a_log"])) * delta
    terms = torch.zeros_like(ry)
    for t in range(0, T, Q):
        e = min(T, t + Q)
        cum = la[t:e].cumsum(0).t()                                                # [H, q]
        m = (c[t:e, 0] @ b[t:e, 0].t()).abs() * torch.exp(cum[:, :, None] - cum[:, None, :]).tril()
        terms[t:e] = ((m * delta[t:e].t()[:, None, :]) @ x[t:e].abs().transpose(0, 1)).transpose(0, 1)
    err = (ref.d(y[0]) - ry).abs()
    assert bool((err <= 2.0 ** -8 * (ry.abs() + terms)).all()), float((err / (ry.abs() + terms)).max())
    assert rel_err(S, rS.numpy(), "fp32") <= SCAN


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_of_more_documents_than_a_block_has_threads(dtype):
    lengths = [(0, 1, 3, 2, 17)[n % 5] for n in range(1100)]
    off = [0, *np.cumsum(lengths).tolist()]
    i, g = ssm_inputs(43, (1, off[-1]), 2, 1, 16, 8, dtype)
    S0 = randn(g, 1100, 2, 16, 8).to(DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True, cu_seqlens=torch.tensor(off, dtype=torch.int32, device=DEV))
    check_scan(i, off, S0, y, S, dtype, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,T", [(3, 6000), (1100, 6000)])
def test_scan_bad_device_offsets_of_long_and_many_documents(dtype, rows, T):
    i, g = ssm_inputs(47, (1, T), 4, 2, 16, 8, dtype)
    S0 = randn(g, rows, 4, 16, 8).to(DEV)
    out = torch.full_like(i["x"], float("nan"))
    cu = torch.linspace(0, T, rows + 1).to(torch.int32)
    cu[1] = cu[2] + 1
    _, S = kda.ssm_scan(*[i[n] for n in ARGS], cu_seqlens=cu.to(DEV), initial_state=S0, output_final_state=True, out=out)
    torch.cuda.synchronize()
    assert kda.device_status() == 1
    assert bool(torch.isnan(out.float()).all()) and torch.equal(S, S0)


def test_scan_is_repeatable_and_runs_on_another_stream():
    i, g = ssm_inputs(23, (1, 3000), 2, 1, 128, 64, "bf16")
    S0 = randn(g, 1, 2, 128, 64).to(DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, S2 = kda.ssm_scan(*[i[n] for n in ARGS], initial_state=S0, output_final_state=True, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(S, S2)


# ------------------------------------------------------------------------------------------- single tokens


def slots_for(B, pool, seed, idle=True):
    rows = torch.from_numpy(np.random.default_rng(seed).permutation(pool)[:B].astype(np.int32))
    if idle and B > 2:
        rows[2] = -1
    return rows


def misaligned(t):
    """The same values one float off the allocation's start."""
    flat = torch.zeros(t.numel() + 1, device=DEV, dtype=t.dtype)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("B,H,G,N,P,dtype,shift", [
    (1, 1, 1, 1, 1, "fp32", False), (5, 4, 2, 64, 64, "bf16", False), (3, 6, 2, 128, 64, "bf16", True),
    (4, 2, 1, 250, 33, "fp32", False), (2, 3, 3, 256, 256, "bf16", False), (7, 4, 1, 48, 40, "fp32", True),
    (3, 2, 1, 20, 100, "bf16", False),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_ssm_step(B, H, G, N, P, dtype, shift, in_place):
    i, g = ssm_inputs(B + N, (B,), H, G, N, P, dtype, strided=True)
    pool = B + 3
    state = randn(g, pool, H, N, P).to(DEV)
    if shift:
        state = misaligned(state)
    slots = slots_for(B, pool, B)
    want_S, want_y = ref.d(state), torch.zeros(B, H, P, dtype=torch.float64)
    for r, s in enumerate(slots.tolist()):
        if s >= 0:
            one = [i[n][r:r + 1] for n in ("x", "dt_raw", "b", "c")]
            y, S = ref.ssm(*one, i["a_log"], i["dt_bias"], i["d_skip"], [0, 1], state[s:s + 1])
            want_y[r], want_S[s] = y[0], S[0]
    out_pool = None if in_place else state.clone()
    before = state.clone()
    y, got = kda.ssm_step(*[i[n] for n in ARGS], state=state, slots=slots.to(DEV), state_out=out_pool)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    assert in_place or torch.equal(state, before)
    assert rel_err(y, want_y.numpy(), dtype) <= (2e-3 if dtype == "bf16" else STEP)
    assert rel_err(got, want_S.numpy(), "fp32") <= STEP
    idle = [s for s in range(pool) if s not in slots.tolist()]
    assert torch.equal(got[idle], before[idle])


def decode_inputs(seed, B, H, Hk, K, V, dtype):
    g = torch.Generator().manual_seed(seed)
    act = lambda *s: randn(g, *s).to(DT[dtype]).to(DEV)  # noqa: E731
    return dict(q=act(B, Hk, K), k=act(B, Hk, K), v=act(B, H, V), g_raw=act(B, H, K), beta_raw=act(B, H),
                a_log=(np.log(16) * torch.rand(H, generator=g)).to(DEV), dt_bias=(0.1 * randn(g, H * K)).to(DEV)), g


DARGS = ("q", "k", "v", "g_raw", "beta_raw", "a_log", "dt_bias")


@pytest.mark.parametrize("B,H,Hk,K,V,dtype,gate,shift", [
    (1, 1, 1, 16, 16, "fp32", "lower_bounded", False), (5, 4, 2, 128, 128, "bf16", "softplus", False),
    (4, 6, 6, 64, 64, "bf16", "lower_bounded", True), (3, 2, 1, 112, 48, "fp32", "softplus", False),
    (6, 3, 3, 48, 112, "bf16", "lower_bounded", False),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_decode_step(B, H, Hk, K, V, dtype, gate, shift, in_place):
    i, g = decode_inputs(B + K, B, H, Hk, K, V, dtype)
    if B > 1:
        i["k"][0] = 0          # a zero key: nothing is written for it
    pool = B + 2
    state = (0.3 * randn(g, pool, H, K, V)).to(DEV)
    if shift:
        state = misaligned(state)
    slots = slots_for(B, pool, B)
    want_S, want_o = ref.d(state), torch.zeros(B, H, V, dtype=torch.float64)
    for r, s in enumerate(slots.tolist()):
        if s >= 0:
            one = [i[n][r] for n in ("q", "k", "v", "g_raw", "beta_raw")]
            want_o[r], want_S[s] = ref.delta_step(*one, i["a_log"], i["dt_bias"], K ** -0.5, -5.0, gate, state[s])
    before = state.clone()
    out, got = kda.decode_step(*[i[n] for n in DARGS], scale=K ** -0.5, gate=gate, state=state, slots=slots.to(DEV),
                               state_out=None if in_place else state.clone())
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    assert in_place or torch.equal(state, before)
    assert rel_err(out, want_o.numpy(), dtype) <= (2e-3 if dtype == "bf16" else STEP)
    assert rel_err(got, want_S.numpy(), "fp32") <= STEP


def test_decode_steps_continue_a_prompt():
    """forward over a prompt, then steps, against forward over all of it (fp32: the step's precision)."""
    B, T, n, H, Hk, K, V = 2, 70, 5, 4, 2, 32, 48
    g = torch.Generator().manual_seed(5)
    act = lambda *s: randn(g, *s).to(DEV)  # noqa: E731
    full = dict(q=act(B, T, Hk, K), k=act(B, T, Hk, K), v=act(B, T, H, V), g_raw=act(B, T, H, K), beta_raw=act(B, T, H))
    par = dict(a_log=(2 * torch.rand(H, generator=g)).to(DEV), dt_bias=act(H * K))
    out, S = kda.forward(*full.values(), *par.values(), scale=K ** -0.5, output_final_state=True)
    head = [t[:, :T - n].contiguous() for t in full.values()]
    _, state = kda.forward(*head, *par.values(), scale=K ** -0.5, output_final_state=True)
    for t in range(T - n, T):
        o, _ = kda.decode_step(*[x[:, t].contiguous() for x in full.values()], *par.values(), scale=K ** -0.5, state=state)
        assert rel_err(o, ref.d(out[:, t]).numpy(), "fp32") <= 1e-4
    assert rel_err(state, ref.d(S).numpy(), "fp32") <= 1e-4


def test_slot_out_of_range_is_reported():
    i, g = ssm_inputs(1, (3,), 2, 1, 32, 32, "bf16")
    state = randn(g, 4, 2, 32, 32).to(DEV)
    before = state.clone()
    y, _ = kda.ssm_step(*[i[n] for n in ARGS], state=state, slots=torch.tensor([4, -3, 1 << 30], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert kda.device_status() == 1
    assert torch.equal(state, before) and not bool(y.any())
    h = torch.zeros(2, 3, 64, device=DEV, dtype=torch.bfloat16)
    yc, _ = kda.short_conv_step(torch.ones(1, 64, device=DEV, dtype=torch.bfloat16), torch.ones(64, 4, device=DEV),
                                history=h, slots=torch.tensor([2], dtype=torch.int32, device=DEV))
    j, g = decode_inputs(1, 1, 2, 2, 32, 32, "bf16")
    s2 = torch.zeros(2, 2, 32, 32, device=DEV)
    o, _ = kda.decode_step(*[j[n] for n in DARGS], scale=1.0, state=s2, slots=torch.tensor([2], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert kda.device_status() == 1
    assert not bool(yc.any()) and not bool(h.any()) and not bool(o.any()) and not bool(s2.any())


# ------------------------------------------------------------------------------------------- convolution


@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("lengths,C,dtype,hist,strided", [
    ([[1]], 8, "fp32", True, False), ([[70], [70]], 64, "bf16", True, True), ([[130]], 1032, "bf16", False, False),
    ([0, 3, 64, 1, 0, 0, 129, 2, 0], 72, "bf16", True, True), ([2, 1, 1, 65], 24, "fp32", True, False),
])
def test_conv_prompt(W, lengths, C, dtype, hist, strided):
    packed = not isinstance(lengths[0], list)
    rows = len(lengths)
    off = [0, *np.cumsum(np.array(lengths).reshape(-1)).tolist()]
    B, T = (1, off[-1]) if packed else (rows, lengths[0][0])
    g = torch.Generator().manual_seed(W + C)
    wide = randn(g, B, T, C + (16 if strided else 0)).to(DT[dtype]).to(DEV)
    x = wide[..., 8:8 + C] if strided else wide
    w, b = randn(g, C, W).to(DEV), randn(g, C).to(DEV)
    h0 = randn(g, rows, W - 1, C).to(DT[dtype]).to(DEV) if hist else None
    cu = torch.tensor(off, dtype=torch.int32, device=DEV) if packed else None
    y, h1 = kda.short_conv_prompt(x, w, b, cu_seqlens=cu, initial_history=h0)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    ry, rh = ref.conv(x.reshape(-1, C), w, b, off, h0)
    assert rel_err(y.reshape(-1, C), ry.numpy(), dtype) <= (2e-3 if dtype == "bf16" else STEP)
    assert torch.equal(ref.d(h1), rh)
    if not packed and h0 is None and not strided:
        assert torch.equal(y, kda.short_conv(x, w, b))


@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("B,C,dtype,in_place", [(1, 8, "fp32", True), (9, 1032, "bf16", False), (300, 64, "bf16", True),
                                                (5, 136, "fp32", False)])
def test_conv_step(W, B, C, dtype, in_place):
    g = torch.Generator().manual_seed(W + B)
    x = randn(g, B, C + 8).to(DT[dtype]).to(DEV)[:, 8:]
    w, b = randn(g, C, W).to(DEV), randn(g, C).to(DEV)
    pool = B + 2
    h = randn(g, pool, W - 1, C).to(DT[dtype]).to(DEV)
    slots = slots_for(B, pool, B)
    want_h, want_y = ref.d(h), torch.zeros(B, C, dtype=torch.float64)
    for r, s in enumerate(slots.tolist()):
        if s >= 0:
            y, last = ref.conv(x[r:r + 1], w, b, [0, 1], h[s:s + 1])
            want_y[r], want_h[s] = y[0], last[0]
    y, got = kda.short_conv_step(x, w, b, history=h, slots=slots.to(DEV), history_out=None if in_place else h.clone())
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    assert rel_err(y, want_y.numpy(), dtype) <= (2e-3 if dtype == "bf16" else STEP)
    assert torch.equal(ref.d(got), want_h)


# ------------------------------------------------------------------------------------------- pages


def cache(seed, S, M, pages, pt, page_bytes, layers=2, lengths=None, spare=0):
    """A cache whose rows hold pages in no order; spare: bytes between the layers, off the pages."""
    rng = np.random.default_rng(seed)
    if lengths is None:
        lengths = rng.integers(0, M * pt + 1, S)
    lengths = np.asarray(lengths, dtype=np.int32)
    order = rng.permutation(pages)
    table, refs, k = np.full((S, M), -1, np.int32), np.zeros(pages, np.int32), 0
    for s in range(S):
        for j in range(-(-int(lengths[s]) // pt)):
            table[s, j] = order[k]
            refs[order[k]] = 1
            k += 1
    wide = torch.from_numpy(rng.integers(0, 256, (layers, pages * page_bytes + spare), dtype=np.uint8)).to(DEV)
    pool = wide[:, :pages * page_bytes].unflatten(1, (pages, page_bytes))
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    return pool, put(table), put(lengths), put(refs)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def same(r, pool, table, lengths, refs):
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    assert np.array_equal(r.table, table.cpu().numpy()) and np.array_equal(r.lengths, lengths.cpu().numpy())
    assert np.array_equal(r.refs, refs.cpu().numpy())
    if pool is not None:
        assert np.array_equal(r.pool, pool.cpu().numpy())


@pytest.mark.parametrize("page_bytes,spare", [(16, 0), (48, 16), (20, 4), (7, 3), (70000, 0)])
@pytest.mark.parametrize("pt", [1, 16, 1 << 30])
@pytest.mark.parametrize("in_place", [True, False])
def test_fork(page_bytes, spare, pt, in_place):
    M = 1 if pt == 1 << 30 else 5
    lengths = {1: [0, 1, 5, 0, 3, 0, 4, 0, 2, 0, 0, 0], 16: [0, 1, 17, 0, 33, 0, 16, 0, 5, 0, 0, 0],
               1 << 30: [0, 9, 1 << 20, 0, 7, 0, 1, 0, 2, 0, 0, 0]}[pt]
    pool, table, lens, refs = cache(1, 12, M, 40 if M > 1 else 16, pt, page_bytes, lengths=lengths, spare=spare)
    r = ref.Cache(pool, table, lens, refs, pt)
    # one parent twice, rows out of range, a child that holds pages, a row onto itself, an empty parent
    parents, children = [2, 2, 4, 8, -1, 12, 1, 6, 4, 10], [0, 3, 5, 7, 9, 9, 6, 6, 99, 11]
    outs = {} if in_place else dict(table_out=torch.full_like(table, 7), lengths_out=torch.full_like(lens, 7),
                                    refs_out=torch.full_like(refs, 7))
    ok = kda.pages_fork(pool, table, lens, refs, ints(*parents), ints(*children), page_tokens=pt, **outs)
    assert ok.cpu().tolist() == r.fork(parents, children) == [1, 1, 1, 1, 0, 0, 0, 0, 0, 1]
    o = outs if outs else dict(table_out=table, lengths_out=lens, refs_out=refs)
    same(r, pool, o["table_out"], o["lengths_out"], o["refs_out"])


def test_fork_until_no_page_is_free():
    pool, table, lens, refs = cache(2, 12, 3, 14, 4, 64, lengths=[5, 9, 4, 0, 0, 0, 0, 0, 0, 0, 0, 0])
    refs[torch.tensor([p for p in range(14) if int(refs[p]) == 0][2:], device=DEV)] = 1     # two pages are left
    r = ref.Cache(pool, table, lens, refs, 4)
    parents, children = [0, 1, 0, 2, 1], [3, 4, 5, 6, 7]
    ok = kda.pages_fork(pool, table, lens, refs, ints(*parents), ints(*children), page_tokens=4)
    assert ok.cpu().tolist() == [1, 1, 0, 1, 0] == r.fork(parents, children)
    same(r, pool, table, lens, refs)


def test_page_ids_out_of_range_are_left_alone():
    pool, table, lens, refs = cache(3, 6, 3, 20, 4, 32, lengths=[9, 9, 12, 0, 0, 0])
    table[0, 2], table[1, 0], table[2, 1] = 20, -5, 1 << 30
    r = ref.Cache(pool, table, lens, refs, 4)
    ok = kda.pages_fork(pool, table, lens, refs, ints(0, 1, 2), ints(3, 4, 5), page_tokens=4)
    assert ok.cpu().tolist() == r.fork([0, 1, 2], [3, 4, 5]) == [0, 1, 1]
    same(r, pool, table, lens, refs)
    kda.pages_free(table, lens, refs, ints(1, 2))
    r.free([1, 2])
    m = kda.pages_compact(pool, table, refs)
    assert np.array_equal(m.cpu().numpy(), r.compact())
    same(r, pool, table, lens, refs)


@pytest.mark.parametrize("in_place", [True, False])
def test_extend(in_place):
    pool, table, lens, refs = cache(4, 9, 4, 22, 8, 16, lengths=[0, 8, 9, 31, 0, 1, 32, 3, 0])
    r = ref.Cache(pool, table, lens, refs, 8)
    # nothing to add, pages to add, shrinking, past the row's end, out of range, more than is left
    seqs, new = [0, 1, 2, 3, 6, 5, 9, 4, 7, 8], [8, 16, 16, 30, 33, 1, 8, 32, 24, 1]
    outs = {} if in_place else dict(table_out=torch.full_like(table, 7), lengths_out=torch.full_like(lens, 7),
                                    refs_out=torch.full_like(refs, 7))
    ok = kda.pages_extend(table, lens, refs, ints(*seqs), ints(*new), page_tokens=8, **outs)
    assert ok.cpu().tolist() == r.extend(seqs, new)
    o = outs if outs else dict(table_out=table, lengths_out=lens, refs_out=refs)
    same(r, None, o["table_out"], o["lengths_out"], o["refs_out"])


def test_extend_refuses_what_does_not_fit():
    pool, table, lens, refs = cache(5, 5, 4, 6, 8, 16, lengths=[8, 0, 0, 0, 0])
    r = ref.Cache(pool, table, lens, refs, 8)
    seqs, new = [1, 2, 3, 0], [24, 32, 8, 8]      # 3 pages, 4 (two are left), 1, none
    ok = kda.pages_extend(table, lens, refs, ints(*seqs), ints(*new), page_tokens=8)
    assert ok.cpu().tolist() == r.extend(seqs, new) == [1, 0, 0, 1]
    same(r, None, table, lens, refs)


@pytest.mark.parametrize("pages,page_bytes", [(50, 16), (50, 12), (9000, 16), (4096, 3)])
@pytest.mark.parametrize("in_place", [True, False])
def test_free_and_compact(pages, page_bytes, in_place):
    S, M = pages // 10, 8
    pool, table, lens, refs = cache(pages, S, M, pages, 4, page_bytes)
    if pages > 1000:
        table[1], lens[1] = table[0].clone(), lens[0].clone()      # two rows on the same pages
        refs.zero_()
        held = table[table >= 0].long()
        refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    r = ref.Cache(pool, table, lens, refs, 4)
    gone = [*range(0, S, 2), S, -1]
    outs = {} if in_place else dict(table_out=torch.full_like(table, 7), lengths_out=torch.full_like(lens, 7),
                                    refs_out=torch.full_like(refs, 7))
    kda.pages_free(table, lens, refs, ints(*gone), **outs)
    r.free(gone)
    if outs:
        table, lens, refs = outs.values()
    same(r, pool, table, lens, refs)
    outs = {} if in_place else dict(table_out=torch.full_like(table, 7), refs_out=torch.full_like(refs, 7))
    m = kda.pages_compact(pool, table, refs, **outs)
    assert np.array_equal(m.cpu().numpy(), r.compact())
    if outs:
        table, refs = outs.values()
    same(r, pool, table, lens, refs)
    m = kda.pages_compact(pool, table, refs)                        # a second time: nothing moves
    assert np.array_equal(m.cpu().numpy(), r.compact())
    same(r, pool, table, lens, refs)


@pytest.mark.parametrize("live", ["none", "all"])
def test_compact_without_moves(live):
    pool, table, lens, refs = cache(6, 4, 4, 16, 4, 16, lengths=[0] * 4 if live == "none" else [16] * 4)
    r = ref.Cache(pool, table, lens, refs, 4)
    m = kda.pages_compact(pool, table, refs)
    assert np.array_equal(m.cpu().numpy(), r.compact())
    same(r, pool, table, lens, refs)


def test_no_requests():
    pool, table, lens, refs = cache(7, 4, 4, 20, 4, 16)
    outs = dict(table_out=torch.full_like(table, 7), lengths_out=torch.full_like(lens, 7), refs_out=torch.full_like(refs, 7))
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert kda.pages_fork(pool, table, lens, refs, none, none, page_tokens=4, **outs).numel() == 0
    torch.cuda.synchronize()
    assert torch.equal(outs["table_out"], table) and torch.equal(outs["refs_out"], refs)
    kda.pages_copy(pool, none, none)
    kda.pages_free(table, lens, refs, none)
    assert kda.device_status() == 0


@pytest.mark.parametrize("page_bytes", [16, 4, 3, 40000])
def test_copy_between_pools(page_bytes):
    a, *_ = cache(8, 1, 1, 12, 4, page_bytes, layers=3)
    b, *_ = cache(9, 1, 1, 7, 4, page_bytes, layers=3, spare=page_bytes)
    want = a.clone()
    src, dst = [0, 6, 3, 7, -1, 2], [5, 0, 11, 1, 2, 12]      # the last three: out of range
    want[:, [5, 0, 11]] = b[:, [0, 6, 3]]
    kda.pages_copy(a, ints(*src), ints(*dst), src_pool=b)
    torch.cuda.synchronize()
    assert torch.equal(a, want)
    want[:, [1, 2]] = a[:, [5, 0]]
    kda.pages_copy(a, ints(5, 0), ints(1, 2))
    torch.cuda.synchronize()
    assert torch.equal(a, want)


def test_binding_refusals():
    i, g = ssm_inputs(1, (2, 8), 4, 2, 16, 16, "bf16")
    bad = [dict(i, b=i["b"][:, :, :, :8]), dict(i, dt_raw=i["dt_raw"].float()), dict(i, a_log=i["a_log"].bfloat16()),
           dict(i, x=i["x"][:, :, :3]), dict(i, d_skip=i["d_skip"][:2])]
    for j in bad:
        with pytest.raises(ValueError):
            kda.ssm_scan(*[j[n] for n in ARGS])
    with pytest.raises(ValueError):
        kda.ssm_scan(*[i[n] for n in ARGS], initial_state=torch.zeros(1, 4, 16, 16, device=DEV))
    with pytest.raises(ValueError):
        kda.ssm_scan(*[i[n] for n in ARGS], cu_seqlens=torch.tensor([0, 16], device=DEV))      # int64
    with pytest.raises(ValueError):
        kda.ssm_scan(*[i[n] for n in ARGS], out=torch.empty(2, 8, 4, 16, device=DEV))
    one = [i[n][:, 0].contiguous() if n in ("x", "b", "c", "dt_raw") else i[n] for n in ARGS]
    for state in (torch.zeros(2, 4, 16, 8, device=DEV), torch.zeros(2, 4, 16, 16, device=DEV, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            kda.ssm_step(*one, state=state)
    with pytest.raises(kda.KdaError):
        kda.ssm_step(*one, state=torch.zeros(1, 4, 16, 16, device=DEV))                         # fewer slots than rows
    with pytest.raises(ValueError):
        kda.ssm_step(*one, state=torch.zeros(2, 4, 16, 16, device=DEV), slots=torch.tensor([0, 1], device=DEV))
    pool, table, lens, refs = cache(7, 4, 4, 20, 4, 16)
    with pytest.raises(ValueError):
        kda.pages_fork(pool[:, :10], table, lens, refs, ints(0), ints(1), page_tokens=4)
    with pytest.raises(ValueError):
        kda.pages_fork(pool, table, lens, refs, ints(0, 1), ints(1), page_tokens=4)
    with pytest.raises(ValueError):
        kda.pages_extend(table.long(), lens, refs, ints(0), ints(1), page_tokens=4)
    with pytest.raises(kda.KdaError):
        kda.pages_extend(table, lens, refs, ints(0), ints(1), page_tokens=0)
