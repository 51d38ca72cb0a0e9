"""GPU tests of the serving operators where a value, an argument or a buffer is unusual.

Tolerances are those of the operators' parity tests unless a test derives its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_delta_rule_sm_gb300 as kda  # noqa: E402
from gated_delta_rule_sm_gb300 import _lib, serve  # noqa: E402
from test_serving import ARGS, DEV, DT, cache, check_scan, ints, randn, run_scan, same, ssm_inputs  # noqa: E402


# ------------------------------------------------------------------------------------------- arguments


@pytest.mark.parametrize("name", ["x", "b", "c", "dt_raw"])
def test_expanded_tokens_are_refused(name):
    i, _ = ssm_inputs(1, (1, 8), 2, 1, 16, 16, "bf16")
    i[name] = i[name][:, :1].expand(i[name].shape)
    with pytest.raises(ValueError):
        kda.ssm_scan(*[i[n] for n in ARGS])
    j, _ = ssm_inputs(1, (8,), 2, 1, 16, 16, "bf16")
    j[name] = j[name][:1].expand(j[name].shape)
    with pytest.raises(ValueError):
        kda.ssm_step(*[j[n] for n in ARGS], state=torch.zeros(8, 2, 16, 16, device=DEV))


def test_expanded_tokens_are_refused_by_the_convolution():
    x, w = torch.zeros(1, 1, 64, device=DEV), torch.zeros(64, 4, device=DEV)
    with pytest.raises(ValueError):
        kda.short_conv_prompt(x.expand(1, 9, 64), w)
    with pytest.raises(ValueError):
        kda.short_conv_step(x[0].expand(9, 64), w, history=torch.zeros(9, 3, 64, device=DEV))


def test_scan_flag_that_raises():
    class Flag:
        def __bool__(self):
            raise ArithmeticError("no truth value")

    i, _ = ssm_inputs(1, (1, 8), 2, 1, 16, 16, "bf16")
    with pytest.raises(ArithmeticError):
        kda.ssm_scan(*[i[n] for n in ARGS], output_final_state=Flag())


# ------------------------------------------------------------------------------------------- scan


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [5, 200, 3001])
def test_scan_with_a_decay_rate_past_fp32(dtype, T):
    """exp(a_log) is infinite in fp32: every token forgets what was before it, also in a row that ends inside a
    block of tokens."""
    i, g = ssm_inputs(51, (1, T), 2, 1, 64, 64, dtype)
    i["a_log"][0] = 100.0
    S0 = randn(g, 1, 2, 64, 64).to(DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True)
    check_scan(i, [0, T], S0, y, S, dtype, dtype == "bf16")


@pytest.mark.parametrize("dtype,N,P,T,docs", [
    ("bf16", 128, 64, 3000, None), ("bf16", 64, 128, 700, None), ("bf16", 64, 64, 420, [70, 0, 150, 200]), ("bf16", 64, 64, 6, None),
    ("fp32", 48, 40, 2100, None), ("fp32", 64, 64, 420, [70, 0, 150, 200]), ("bf16", 256, 64, 300, None),
])
def test_scan_in_place(dtype, N, P, T, docs):
    """y over x and the end states over the entering ones give what separate buffers give."""
    i, g = ssm_inputs(53, (1, T), 4, 2, N, P, dtype)
    cu = None if docs is None else torch.tensor([0, *np.cumsum(docs).tolist()], dtype=torch.int32, device=DEV)
    S0 = randn(g, len(docs) if docs else 1, 4, N, P).to(DEV)
    y, S = run_scan(i, initial_state=S0, output_final_state=True, cu_seqlens=cu)
    for _ in range(3):
        x, state = i["x"].clone(), S0.clone()
        y2, S2 = run_scan(dict(i, x=x), initial_state=state, output_final_state=True, cu_seqlens=cu, out=x, final_state=state)
        assert y2 is x and S2 is state
        assert torch.equal(y, x) and torch.equal(S, state)


# ------------------------------------------------------------------------------------------- convolution


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("step", [False, True])
def test_conv_far_below_zero(dtype, step):
    """y = a sigmoid(a) tends to zero as a falls, and is -inf * 0 at -inf; each value beside an ordinary one.

    fp32: the exponent of 2 is up to 60 and rounded to 2^-24 of itself, which is 2.5e-6 of the exponential, and a
    few roundings follow: 1e-5.  Below a = -60 ln 2 the result may be 0, which is 60 ln 2 / 2^60 = 4e-17 off."""
    low = [-30.0, -40.0, -41.0, -42.0, -50.0, -64.0, -88.0, -1e3, -1e12, -1e20, -3e38, float("-inf")]
    a = torch.tensor([v for i, x in enumerate(low) for v in ((x, 0.7 - i) if i % 2 else (i - 5.3, x))]).to(DT[dtype])
    C = a.numel()
    assert C % 8 == 0
    w = torch.zeros(C, 4)
    w[:, 3] = 1.0
    if step:
        h = torch.zeros(1, 3, C, dtype=DT[dtype], device=DEV)
        y, _ = kda.short_conv_step(a[None].to(DEV), w.to(DEV), history=h)
    else:
        y, _ = kda.short_conv_prompt(a[None, None].to(DEV), w.to(DEV))
    torch.cuda.synchronize()
    y, want = ref.d(y).flatten(), ref.d(a) * torch.sigmoid(ref.d(a))
    nan = torch.isnan(want)
    assert int(nan.sum()) == 1 and torch.equal(torch.isnan(y), nan)
    rel = 2.0 ** -8 if dtype == "bf16" else 1e-5
    err = (y - want).abs()[~nan]
    assert bool((err <= rel * want.abs()[~nan] + 1e-16).all()), (err - rel * want.abs()[~nan]).max()


@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype,C", [("bf16", 1032), ("fp32", 64)])
@pytest.mark.parametrize("lengths", [[1] * 5, [0, 3, 2000, 1, 0, 0, 7, 2, 5, 600, 0], [1500] * 3])
def test_conv_history_in_place(W, dtype, C, lengths):
    """final_history over initial_history gives what separate buffers give: rows shorter than the window,
    empty ones, and rows that many CTAs read."""
    rows, T = len(lengths), sum(lengths)
    g = torch.Generator().manual_seed(T + W)
    x = randn(g, 1, T, C).to(DT[dtype]).to(DEV)
    w, h = randn(g, C, W).to(DEV), randn(g, rows, W - 1, C).to(DT[dtype]).to(DEV)
    cu = torch.tensor([0, *np.cumsum(lengths).tolist()], dtype=torch.int32, device=DEV)
    y, last = kda.short_conv_prompt(x, w, cu_seqlens=cu, initial_history=h)
    for _ in range(5):
        k = h.clone()
        y2, last2 = kda.short_conv_prompt(x, w, cu_seqlens=cu, initial_history=k, final_history=k)
        assert last2 is k
        assert torch.equal(y, y2) and torch.equal(last, k)
    assert kda.device_status() == 0


# ------------------------------------------------------------------------------------------- pages


def many(*v):
    return torch.tensor(np.asarray(v).reshape(-1), dtype=torch.int32, device=DEV)


def outputs(table, lens, refs, in_place):
    if in_place:
        return {}
    return dict(table_out=torch.full_like(table, 7), lengths_out=torch.full_like(lens, 7), refs_out=torch.full_like(refs, 7))


# one pass over the pages (up to 16384 of them) with several tiles, and two passes; the free pages lie in all tiles
@pytest.mark.parametrize("pages", [5000, 9000, 16384, 16385, 40000])
@pytest.mark.parametrize("in_place", [True, False])
def test_fork_and_extend_over_many_tiles(pages, in_place):
    S, M, pt = pages // 4, 8, 4
    rng = np.random.default_rng(pages)
    lengths = rng.integers(1, M * pt + 1, S)
    children = rng.permutation(S)[:S // 3]
    lengths[children] = 0
    pool, table, lens, refs = cache(pages, S, M, pages, pt, 8, layers=2, lengths=lengths)
    r = ref.Cache(pool, table, lens, refs, pt)
    others = np.append(np.setdiff1d(np.arange(S), children), [-1, S])
    parents = rng.choice(others, len(children))
    o = outputs(table, lens, refs, in_place)
    ok = kda.pages_fork(pool, table, lens, refs, many(parents), many(children), page_tokens=pt, **o)
    assert ok.cpu().tolist() == r.fork(parents.tolist(), children.tolist())
    if o:
        table, lens, refs = o["table_out"], o["lengths_out"], o["refs_out"]
    same(r, pool, table, lens, refs)
    # more than the pages that are left: the last requests are refused
    seqs = rng.permutation(S)
    new = np.minimum(r.lengths[seqs] + rng.integers(0, 2 * M * pt, S), M * pt + 1)
    o = outputs(table, lens, refs, in_place)
    ok = kda.pages_extend(table, lens, refs, many(seqs), many(new), page_tokens=pt, **o).cpu().tolist()
    assert ok == r.extend(seqs.tolist(), new.tolist()) and 0 < sum(ok) < len(ok)
    if o:
        table, lens, refs = o["table_out"], o["lengths_out"], o["refs_out"]
    same(r, None, table, lens, refs)


@pytest.mark.parametrize("pages,page_bytes", [(16384, 16), (16385, 4), (40000, 16)])
@pytest.mark.parametrize("in_place", [True, False])
def test_free_and_compact_over_many_tiles(pages, page_bytes, in_place):
    S, M = pages // 10, 8
    pool, table, lens, refs = cache(pages, S, M, pages, 4, page_bytes, layers=2)
    r = ref.Cache(pool, table, lens, refs, 4)
    gone = np.random.default_rng(1).permutation(S)[:S // 2]
    o = outputs(table, lens, refs, in_place)
    kda.pages_free(table, lens, refs, many(gone), **o)
    r.free(gone.tolist())
    if o:
        table, lens, refs = o["table_out"], o["lengths_out"], o["refs_out"]
    same(r, pool, table, lens, refs)
    o = outputs(table, lens, refs, in_place)
    o.pop("lengths_out", None)
    m = kda.pages_compact(pool, table, refs, **o)
    assert np.array_equal(m.cpu().numpy(), r.compact())
    if o:
        table, refs = o["table_out"], o["refs_out"]
    same(r, pool, table, lens, refs)


def test_more_requests_than_a_block_has_threads():
    """Ranks carry on from one 1024 requests to the next; the pages run out in the third."""
    S, M, pt = 3000, 2, 4
    lengths = np.where(np.arange(S) < 400, 5, 0)
    pool, table, lens, refs = cache(3, S, M, 3000, pt, 4, lengths=lengths)
    r = ref.Cache(pool, table, lens, refs, pt)
    parents, children = np.arange(2600) % 400, np.arange(400, 3000)
    ok = kda.pages_fork(pool, table, lens, refs, many(parents), many(children), page_tokens=pt).cpu().tolist()
    assert ok == r.fork(parents.tolist(), children.tolist()) and 2048 < sum(ok) < 2600
    same(r, pool, table, lens, refs)
    pool, table, lens, refs = cache(4, S, M, 2300, pt, 4, lengths=[0] * S)
    r = ref.Cache(pool, table, lens, refs, pt)
    new = [1 + (n % 7 == 0) * 4 for n in range(2600)]
    ok = kda.pages_extend(table, lens, refs, many(np.arange(2600)), many(new), page_tokens=pt).cpu().tolist()
    assert ok == r.extend(list(range(2600)), new) and 0 < sum(ok) < 2600
    same(r, None, table, lens, refs)


def test_extend_of_a_row_named_twice_stays_in_its_row():
    """Against the contract, but known to the device only: nothing outside the row is written."""
    S, M, pt = 4, 6, 4
    for _ in range(20):
        wide = torch.full((S + 2, M), -1, dtype=torch.int32, device=DEV)
        lens = torch.zeros(S, dtype=torch.int32, device=DEV)
        refs = torch.zeros(64, dtype=torch.int32, device=DEV)
        kda.pages_extend(wide[:S], lens, refs, ints(*[S - 1] * 8, 0), ints(*[M * pt] * 8, 5), page_tokens=pt)
        rows = wide.tolist()
        assert rows[1:S - 1] == [[-1] * M] * (S - 2) and rows[S:] == [[-1] * M] * 2
        assert all(0 <= p < 64 for p in rows[S - 1]) and lens.tolist() == [5, 0, 0, M * pt]
        assert rows[0][2:] == [-1] * (M - 2)


# ------------------------------------------------------------------------------------------- captured calls


def test_captured_calls_keep_their_workspaces():
    """A graph's workspaces are its own: later calls on its stream that want more do not take them away, and its
    replays write nobody else's memory."""
    small, _ = ssm_inputs(61, (1, 3000), 2, 1, 64, 64, "bf16")
    large, _ = ssm_inputs(62, (1, 9000), 4, 1, 64, 64, "bf16")
    pool, table, lens, refs = cache(3, 6, 4, 40, 4, 64, lengths=[9, 5, 1, 0, 0, 0])
    outs = [torch.empty_like(t) for t in (table, lens, refs)]
    kw = dict(page_tokens=4, table_out=outs[0], lengths_out=outs[1], refs_out=outs[2])
    parents, children = ints(0, 1), ints(3, 4)
    side = torch.cuda.Stream()
    _lib.workspace_cache.clear()       # (earlier tests' calls on this stream may have wanted more)

    def calls():
        y, S = kda.ssm_scan(*[small[n] for n in ARGS], output_final_state=True)
        return y, S, kda.pages_fork(pool, table, lens, refs, parents, children, **kw), *outs

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in calls()]
    side.synchronize()
    kept = {k: (t.data_ptr(), t.numel()) for k, t in _lib.workspace_cache.buf.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = calls()
    assert {k: (t.data_ptr(), t.numel()) for k, t in _lib.workspace_cache.buf.items()} == kept
    with torch.cuda.stream(side):
        kda.ssm_scan(*[large[n] for n in ARGS], output_final_state=True)       # wants more
        sizes = [n for _, n in kept.values()]
        others = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
        for t in outs:
            t.fill_(99)
        graph.replay()
        graph.replay()
    side.synchronize()
    assert max(t.numel() for t in _lib.workspace_cache.buf.values()) > max(sizes)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 7).all()) for t in others)
    assert kda.device_status() == 0


def test_first_call_on_a_stream_may_be_captured():
    i, _ = ssm_inputs(63, (1, 3000), 2, 1, 64, 64, "bf16")
    want, _ = kda.ssm_scan(*[i[n] for n in ARGS])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    before = set(_lib.workspace_cache.buf)
    with torch.cuda.graph(graph, stream=side):
        got, _ = kda.ssm_scan(*[i[n] for n in ARGS])
    assert set(_lib.workspace_cache.buf) == before
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and kda.device_status() == 0


# ------------------------------------------------------------------------------------------- the served decoder


def test_refused_fork_leaves_every_pool():
    """A child that still holds its page keeps it, in every layer's pools; the other request is served."""
    model = serve.Decoder(layers=2, heads=2, groups=1, dim=32, head_dim=16, state_dim=16)
    cch = serve.StateCache(model, slots=6, sequences=4)
    assert cch.admit(ints(0, 1), ints(5, 9)).tolist() == [1, 1]
    for k, pool in enumerate(cch.every_pool()):
        pool.copy_(torch.randn(pool.shape, generator=torch.Generator().manual_seed(k)).to(pool.dtype))
    before = [pool.clone() for pool in cch.every_pool()]
    held, parent = cch.slots(ints(1)).item(), cch.slots(ints(0)).item()
    assert cch.fork(ints(0, 0), ints(1, 2)).tolist() == [0, 1]
    child = cch.slots(ints(2)).item()
    assert cch.slots(ints(1)).item() == held and child not in (held, parent)
    for pool, old in zip(cch.every_pool(), before):
        old[:, child] = old[:, parent]
        assert torch.equal(pool, old)
    assert kda.device_status() == 0
