"""GPU parity of attention over paged keys and values, and of what writes them, against plain 64-bit references.

Tolerances, derived before the first run.  Written keys and values are equal.  An output is sum w v: with relative errors
e of the weights it is off by up to e sum w |v|, which the reference gives.
  * bf16: the weights are rounded to bf16 before they meet the values (2^-8) while their sum is not, and the output is rounded
    once (2^-8 |out|); scores are fp32 sums of exact products: (2^-8 + 1e-4) sum w |v| + 2^-8 |out|;
  * fp32: a score is a sum of D products, off by up to about sqrt(D) 2^-24 of sum |q k| < 2^-20 * 40 here, and with it the
    exponential: 1e-4 sum w |v| leaves a margin of two;
  * lse: the scores' error, 1e-4, and a few roundings of the result, 1e-6 |lse|."""
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

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Case:
    """Sequences of `held` tokens, of which the last `new` are this call's; table rows and pages in no order."""

    def __init__(self, held, new, Hq, Hkv, D, pt, dtype, seed=0, spare=3, seqs=None, dirty=True):
        g = torch.Generator().manual_seed(seed)
        self.g, self.new, self.Hq, self.Hkv, self.D, self.pt, self.dtype = g, new, Hq, Hkv, D, pt, dtype
        rows, need = len(held), [-(-n // pt) for n in held]
        order = torch.randperm(rows + 1, generator=g)[:rows].tolist()
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((rows + 1, max(1, max(need))), -1, dtype=torch.int32)
        self.lengths = torch.zeros(rows + 1, dtype=torch.int32)
        for r in range(rows):
            for j in range(need[r]):
                self.table[order[r], j] = perm.pop()
            self.lengths[order[r]] = held[r]
        self.seqs = torch.tensor(order if seqs is None else seqs(order), dtype=torch.int32)
        self.pool = torch.randn(pages, 2, Hkv, pt, D, generator=g).to(DT[dtype])
        if dirty:        # what no token of the cache holds is NaN
            live = torch.zeros(pages, pt, dtype=torch.bool)
            for r in range(rows):
                for p in range(held[r]):
                    live[self.table[order[r], p // pt], p % pt] = True
            self.pool.permute(0, 3, 1, 2, 4)[~live] = float("nan")
        self.off = [0, *np.cumsum(new).tolist()]
        self.q = torch.randn(self.off[-1], Hq, D, generator=g).to(DT[dtype])

    def packed(self):
        return dict(seqs=self.seqs.to(DEV), cu_seqlens=ints(self.off))

    def run(self, window=0, scale=None, q=None, lse=True, packed=True, **kw):
        scale = self.D ** -0.5 if scale is None else scale
        q = self.q.to(DEV)[None] if q is None else q
        args = self.packed() if packed else dict(seqs=self.seqs.to(DEV))
        lse = torch.full(q.shape[:3], 5.0, device=DEV) if lse else None
        out = kda.pages_attention(q, self.pool.to(DEV), self.table.to(DEV), self.lengths.to(DEV), scale=scale, window=window, lse=lse, **args, **kw)
        torch.cuda.synchronize()
        assert kda.device_status() == 0
        return out, lse

    def check(self, out, lse, window=0, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        want, size, wl = ref.attention(self.q, self.pool, self.table, self.lengths, self.seqs, self.off, scale, window)
        w = 2.0 ** -8 + 1e-4 if self.dtype == "bf16" else 1e-4
        store = 2.0 ** -8 if self.dtype == "bf16" else 0.0
        err = (ref.d(out).reshape(want.shape) - want).abs() - (w * size + store * want.abs() + 1e-30)
        assert bool((err <= 0).all()), float(err.max())
        empty = wl == -np.inf
        assert not bool(out.reshape(want.shape).cpu()[empty].any())
        if lse is not None:
            mine = ref.d(lse).reshape(wl.shape)
            assert bool((mine[empty] == -np.inf).all())
            if not bool(empty.all()):
                assert bool(((mine[~empty] - wl[~empty]).abs() <= 1e-4 + 1e-6 * wl[~empty].abs()).all())


# a token a row: lengths around pages and tiles, empty and idle rows; heads of every group size; sizes of every kernel
@pytest.mark.parametrize("Hq,Hkv,D,pt,dtype", [
    (8, 2, 128, 16, "bf16"), (4, 4, 64, 16, "bf16"), (16, 1, 128, 64, "bf16"), (6, 2, 96, 24, "bf16"), (5, 1, 40, 1, "bf16"),
    (32, 1, 128, 16, "bf16"), (40, 1, 64, 7, "bf16"), (2, 1, 256, 16, "bf16"), (3, 3, 200, 5, "bf16"), (3, 3, 33, 16, "bf16"), (2, 2, 8, 128, "bf16"),
    (4, 2, 128, 16, "fp32"), (3, 1, 40, 24, "fp32"), (2, 1, 250, 3, "fp32"),
])
@pytest.mark.parametrize("window", [0, 33])
def test_one_token_a_row(Hq, Hkv, D, pt, dtype, window):
    held = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 0, 31, 1000]
    c = Case(held, [1] * len(held), Hq, Hkv, D, pt, dtype, seed=D + pt, seqs=lambda o: [-1 if r == 4 else s for r, s in enumerate(o)])
    out, lse = c.run(window, q=c.q.to(DEV)[:, None], packed=False)
    c.check(out, lse, window)
    # packed, the same
    out2, lse2 = c.run(window)
    assert torch.equal(out2[0], out[:, 0]) and torch.equal(lse2[0], lse[:, 0])


@pytest.mark.parametrize("Hq,Hkv,D,pt,dtype", [
    (8, 2, 128, 16, "bf16"), (4, 4, 64, 16, "bf16"), (6, 2, 96, 24, "bf16"), (5, 1, 40, 1, "bf16"), (16, 1, 128, 64, "bf16"), (7, 1, 72, 10, "bf16"),
    (2, 1, 256, 16, "bf16"), (3, 3, 33, 16, "bf16"), (4, 2, 128, 16, "fp32"), (3, 1, 40, 24, "fp32"), (2, 2, 256, 5, "fp32"),
])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_chunks(Hq, Hkv, D, pt, dtype, window):
    """Chunks of new tokens over what was there: none, one, around a block of rows and a tile of keys; a row without tokens."""
    new = [1, 0, 16, 63, 130, 5, 300, 33]
    past = [0, 9, 100, 1, 250, 700, 0, 128]
    held = [p + n for p, n in zip(past, new)]
    c = Case(held, new, Hq, Hkv, D, pt, dtype, seed=D, seqs=lambda o: [-1 if r == 5 else s for r, s in enumerate(o)])
    c.check(*c.run(window), window)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
@pytest.mark.parametrize("new", [1, 3, 50, 260])
def test_long_rows_are_cut_and_joined(dtype, D, new):
    """Few rows over many keys: every CTA takes a part."""
    c = Case([9000, 4100], [new, 1], 8, 2, D, 16, dtype, seed=new, dirty=False)
    c.check(*c.run())
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*c.run(window=5000), window=5000)


@pytest.mark.parametrize("Hq,Hkv,D,pt,dtype,new", [
    (8, 2, 128, 16, "bf16", 3), (8, 2, 128, 16, "bf16", 8), (8, 2, 128, 16, "bf16", 9), (4, 1, 64, 8, "bf16", 64), (4, 1, 64, 8, "bf16", 65),
    (2, 1, 256, 16, "bf16", 8), (2, 1, 256, 16, "bf16", 9), (4, 2, 64, 16, "fp32", 32), (4, 2, 64, 16, "fp32", 33),
])
def test_as_many_new_tokens_in_every_row(Hq, Hkv, D, pt, dtype, new):
    """Without offsets, around the sizes at which a row stops being one block; a window that no position reaches is none."""
    c = Case([new + p for p in (0, 1, 77, 300, 3, 900)], [new] * 6, Hq, Hkv, D, pt, dtype, seed=new, seqs=lambda o: [-1 if r == 4 else s for r, s in enumerate(o)])
    q = c.q.to(DEV).reshape(6, new, Hq, D)
    out, lse = c.run(q=q, packed=False)
    c.check(out.reshape(1, -1, Hq, D), lse.reshape(1, -1, Hq))
    out2, lse2 = c.run(2 ** 31 - 1, q=q, packed=False)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G,n,dtype", [(4, 1, "bf16"), (16, 2, "bf16"), (4, 1, "fp32")])
def test_more_rows_than_a_cta_counts_for_itself(G, n, dtype):
    """The plan's launch, for rows of one block each: lengths around a page, every ninth row idle, others without a token yet."""
    rows = 601
    held = [0 if r % 7 == 3 else n + r % 40 for r in range(rows)]
    c = Case(held, [n] * rows, G, 1, 64, 16, dtype, seed=n, seqs=lambda o: [-1 if r % 9 == 5 else s for r, s in enumerate(o)])
    q = c.q.to(DEV).reshape(rows, n, G, 64)
    out, lse = c.run(q=q, packed=False)
    c.check(out.reshape(1, -1, G, 64), lse.reshape(1, -1, G))


def test_a_chunk_longer_than_its_sequence():
    """Tokens at negative positions have no keys: zeros, and they are not written."""
    for dtype in ("bf16", "fp32"):
        c = Case([3, 40], [10, 20], 4, 2, 64, 16, dtype)
        c.check(*c.run())
        k, v = torch.randn(30, 2, 64, generator=c.g).to(DT[dtype]), torch.randn(30, 2, 64, generator=c.g).to(DT[dtype])
        pool = c.pool.to(DEV)
        kda.pages_append(pool, c.table.to(DEV), c.lengths.to(DEV), k.to(DEV)[None], v.to(DEV)[None], **c.packed())
        want = ref.append(c.pool, c.table, c.lengths, k, v, c.seqs, c.off)
        assert torch.equal(pool.cpu().nan_to_num(77.0), want.nan_to_num(77.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scores_at_their_ends(dtype):
    """Large scores of both signs, equal scores, a scale of zero: the largest score's exponential is 1 whatever its size."""
    c = Case([300, 70], [40, 1], 4, 2, 64, 16, dtype, dirty=False)
    c.check(*c.run(scale=0.0), scale=0.0)
    c.pool[:, 0] *= 0
    c.check(*c.run())
    c = Case([300, 70], [40, 1], 4, 2, 64, 16, dtype, dirty=False)
    c.pool[:, 0] = torch.sign(c.pool[:, 0].float()).to(c.pool.dtype)      # whole scores: exact in both types, up to +-64 * 200
    c.q = torch.sign(c.q.float()).to(c.q.dtype)
    c.check(*c.run(scale=200.0), scale=200.0)
    c.check(*c.run(scale=-200.0), scale=-200.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new", [[1, 1, 1], [70, 3, 200]])
def test_rows_untouched_by_others(dtype, new):
    """NaN in every page of other sequences, and in keys that the mask hides, leave a row as it was."""
    c = Case([200, 90, 333], new, 8, 2, 128, 16, dtype, seed=2)
    out, lse = c.run(window=150)
    want = out[0, c.off[1]:c.off[2]].clone()
    for r in (0, 2):
        for page in c.table[c.seqs[r]].tolist():
            if page >= 0:
                c.pool[page] = float("nan")
    out, lse = c.run(window=150)
    assert torch.equal(out[0, c.off[1]:c.off[2]], want)
    # a key that is NaN at the newest position is seen by the last token alone
    if new[1] > 1:
        p = 89
        c.pool[c.table[c.seqs[1], p // 16], 0, :, p % 16] = float("nan")
        out, lse = c.run(window=150)
        got = out[0, c.off[1]:c.off[2]]
        assert torch.equal(got[:-1], want[:-1]) and bool(torch.isnan(got[-1]).all())


def test_a_page_that_is_not_one():
    """Recorded, and its keys count as zeros; what is past the length is not looked at."""
    for dtype in ("bf16", "fp32"):
        for new in (1, 40):
            c = Case([200, 100], [new, new], 4, 2, 64, 16, dtype, dirty=False)
            want, _ = c.run()
            c.table[c.seqs[1], 7:] = -5                          # past 100 tokens: seven pages
            again, _ = c.run()
            assert torch.equal(want, again)
            for bad in (-1, c.pool.shape[0], 1 << 30):
                broken = c.table.clone()
                broken[c.seqs[0], 2] = bad
                out = kda.pages_attention(c.q.to(DEV)[None], c.pool.to(DEV), broken.to(DEV), c.lengths.to(DEV), scale=0.125, **c.packed())
                assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG
                assert bool(torch.isfinite(out).all()) and torch.equal(out[0, new:], want[0, new:])
                pool = c.pool.to(DEV)
                k = torch.randn(1, 2 * new, 2, 64, generator=c.g).to(DT[dtype]).to(DEV)
                broken[c.seqs[0], 12] = bad                       # position 199
                kda.pages_append(pool, broken.to(DEV), c.lengths.to(DEV), k, k, **c.packed())
                assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG


def test_rows_and_lengths_past_the_table():
    c = Case([50, 60], [1, 1], 4, 2, 64, 16, "bf16", dirty=False)
    want, _ = c.run()
    for seqs, lengths in ((ints([int(c.seqs[0]), 99]), c.lengths), (c.seqs.to(DEV), c.lengths.clone().index_fill_(0, c.seqs[1:].long(), 1000))):
        out = kda.pages_attention(c.q.to(DEV)[None], c.pool.to(DEV), c.table.to(DEV), lengths.to(DEV), scale=0.125, seqs=seqs, cu_seqlens=ints(c.off))
        assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG
        assert torch.equal(out[0, 0], want[0, 0]) and not bool(out[0, 1].any())
        pool = c.pool.to(DEV)
        k = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16, device=DEV)
        kda.pages_append(pool, c.table.to(DEV), lengths.to(DEV), k, k, seqs=seqs, cu_seqlens=ints(c.off))
        assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG
        page, at = c.table[c.seqs[1], 59 // 16], 59 % 16
        assert torch.equal(pool[page, :, :, at].cpu(), c.pool[page, :, :, at])


def test_offsets_that_break_the_contract():
    c = Case([50, 60], [10, 20], 4, 2, 64, 16, "bf16", dirty=False)
    for bad in ([0, 10, 29], [1, 10, 30], [0, 31, 30]):
        out = torch.full((1, 30, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
        args = (c.pool.to(DEV), c.table.to(DEV), c.lengths.to(DEV))
        kda.pages_attention(c.q.to(DEV)[None], *args, scale=0.125, seqs=c.seqs.to(DEV), cu_seqlens=ints(bad), out=out)
        assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG and bool((out == 3.0).all())
        k = torch.zeros(1, 30, 2, 64, dtype=torch.bfloat16, device=DEV)
        kda.pages_append(*args, k, k, seqs=c.seqs.to(DEV), cu_seqlens=ints(bad))
        assert kda.device_status() == _lib.KDA_ERR_INVALID_ARG and torch.equal(args[0].cpu(), c.pool)
        with pytest.raises(kda.KdaError):
            kda.pages_attention(c.q.to(DEV)[None], *args, scale=0.125, seqs=c.seqs.to(DEV), cu_seqlens=ints(bad), cu_seqlens_host=bad)


@pytest.mark.parametrize("Hkv,D,pt,dtype", [(2, 128, 16, "bf16"), (8, 64, 24, "bf16"), (3, 33, 16, "bf16"), (1, 8, 1, "bf16"), (5, 256, 7, "fp32"), (2, 3, 16, "fp32")])
@pytest.mark.parametrize("strided", [False, True])
def test_append(Hkv, D, pt, dtype, strided):
    new = [1, 0, 16, 63, 130, 5]
    held = [p + n for p, n in zip([0, 9, 100, 1, 250, 70], new)]
    c = Case(held, new, Hkv, Hkv, D, pt, dtype, seed=D, seqs=lambda o: [-1 if r == 3 else s for r, s in enumerate(o)])
    kv = torch.randn(sum(new), 2 * Hkv * D + 8, generator=c.g).to(DT[dtype])
    k, v = kv[:, :Hkv * D].unflatten(1, (Hkv, D)), kv[:, Hkv * D:2 * Hkv * D].unflatten(1, (Hkv, D))
    want = ref.append(c.pool, c.table, c.lengths, k, v, c.seqs, c.off)
    dev = kv.to(DEV)
    dk, dv = dev[:, :Hkv * D].unflatten(1, (Hkv, D))[None], dev[:, Hkv * D:2 * Hkv * D].unflatten(1, (Hkv, D))[None]
    if not strided:
        dk, dv = dk.contiguous(), dv.contiguous()
    pool = c.pool.to(DEV)
    assert kda.pages_append(pool, c.table.to(DEV), c.lengths.to(DEV), dk, dv, **c.packed()) is pool
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    assert torch.equal(pool.cpu().nan_to_num(77.0), want.nan_to_num(77.0))


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 40)])
@pytest.mark.parametrize("new", [1, 37])
def test_slices_and_given_results(dtype, D, new):
    c = Case([100, 50], [new, new], 4, 2, D, 16, dtype)
    want, wl = c.run()
    for off in (0, 1, 8):         # a slice that 16-byte pieces reach, and ones that they do not
        wide = torch.randn(2 * new, 4 * D + 16, generator=c.g).to(DT[dtype]).to(DEV)
        wide[:, off:off + 4 * D] = c.q.to(DEV).flatten(1)
        q = wide[:, off:off + 4 * D].unflatten(1, (4, D))[None]
        out = torch.full((1, 2 * new, 4, D), 3.0, dtype=DT[dtype], device=DEV)
        got, lse = c.run(q=q, out=out)
        assert got is out
        c.check(out, lse)
    flat = torch.zeros(c.pool.numel() + 1, dtype=DT[dtype], device=DEV)      # a pool at an odd element
    flat[1:] = c.pool.to(DEV).reshape(-1)
    out = kda.pages_attention(c.q.to(DEV)[None], flat[1:].view(c.pool.shape), c.table.to(DEV), c.lengths.to(DEV), scale=D ** -0.5, **c.packed())
    c.check(out, None)


def test_a_pool_past_32_bits():
    """Pages whose elements' indices pass 2^31 and whose bytes pass 2^32."""
    pages, pt, Hkv, D = 66000, 16, 8, 128                # 4.3 GB; a page 64 KB
    pool = torch.zeros(pages, 2, Hkv, pt, D, dtype=torch.bfloat16, device=DEV)
    table = ints([[pages - 1, 3, pages - 2]])
    lengths = ints([40])
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, 40, Hkv, D, generator=g).bfloat16() for _ in range(2))
    kda.pages_append(pool, table, lengths, k.to(DEV), v.to(DEV), cu_seqlens=ints([0, 40]))
    assert torch.equal(pool[pages - 2, 0, :, 7].cpu(), k[0, 39]) and torch.equal(pool[pages - 1, 1, :, 15].cpu(), v[0, 15])
    small = pool[[pages - 1, 3, pages - 2]].cpu()
    for n in (1, 40):
        q = torch.randn(n, Hkv, D, generator=g).bfloat16()
        out = kda.pages_attention(q.to(DEV)[None], pool, table, lengths, scale=0.1)
        want, size, _ = ref.attention(q, small, torch.tensor([[0, 1, 2]]), torch.tensor([40]), [0], [0, n], 0.1, 0)
        assert bool(((ref.d(out[0]) - want).abs() <= (2.0 ** -8 + 1e-4) * size + 2.0 ** -8 * want.abs()).all())
    assert kda.device_status() == 0


def test_streams_and_captured_graphs():
    cases = [Case([3000, 700, 90], [1, 1, 1], 8, 2, 128, 16, "bf16", seed=s, dirty=False) for s in (1, 2)]
    chunks = [Case([3000, 700], [200, 300], 8, 2, 128, 16, "bf16", seed=s, dirty=False) for s in (3, 4)]
    dev = [(c.q.to(DEV)[None], c.pool.to(DEV), c.table.to(DEV), c.lengths.to(DEV), c.packed()) for c in cases + chunks]
    call = lambda d, **kw: kda.pages_attention(*d[:4], scale=0.1, **d[4], **kw)  # noqa: E731
    want = [call(d) for d in dev]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [call(dev[k % 4], stream=streams[k % 2]) for k in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[k % 4]) for k, t in enumerate(got))
    graphs, outs = [], []
    for d in dev:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(d))
        graphs.append(graph)
    for k in (0, 1, 2):
        for o in outs:
            o.fill_(9.0)
        torch.cuda.synchronize()
        graphs[k].replay()
        with torch.cuda.stream(streams[0]):
            graphs[k + 1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[k], want[k]) and torch.equal(outs[k + 1], want[k + 1])
    # a captured step follows lengths that grow in place
    d, c = dev[0], cases[0]
    d[3][c.seqs.long()] -= 1
    c.lengths[c.seqs.long()] -= 1
    graphs[0].replay()
    torch.cuda.synchronize()
    c.check(outs[0], None, scale=0.1)


def test_calls_of_several_host_threads():
    """The C entry from four threads at once, head sizes of one kernel among them, each on its own stream with its own workspace."""
    import ctypes
    import threading
    lib = _lib.load()
    cases = [Case([400, 90], [30, 1], 4, 2, D, 16, dtype, seed=D, dirty=False) for D, dtype in ((40, "fp32"), (64, "fp32"), (250, "fp32"), (33, "bf16"))]
    args = []
    for c in cases:
        t = dict(q=c.q.to(DEV), pool=c.pool.to(DEV), table=c.table.to(DEV), lengths=c.lengths.to(DEV), seqs=c.seqs.to(DEV), cu=ints(c.off))
        dims = _lib.AttentionDims(rows=2, tokens=31, Hq=4, Hkv=2, D=c.D, dtype=_lib.KDA_BF16 if c.dtype == "bf16" else _lib.KDA_FP32, num_pages=c.pool.shape[0],
                                  page_tokens=16, table_rows=c.table.shape[0], max_pages=c.table.shape[1])
        ws = torch.empty(lib.kda_pages_attention_workspace_size(ctypes.byref(dims)), dtype=torch.uint8, device=DEV)
        args.append((dims, t, ws, torch.zeros(31, 4, c.D, dtype=DT[c.dtype], device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    said, gate = [], threading.Barrier(len(args))

    def work(dims, t, ws, out, stream):
        gate.wait()
        for _ in range(50):
            said.append(lib.kda_pages_attention(ctypes.byref(dims), t["q"].data_ptr(), t["pool"].data_ptr(), t["table"].data_ptr(), t["lengths"].data_ptr(),
                                                t["seqs"].data_ptr(), t["cu"].data_ptr(), None, dims.D ** -0.5, out.data_ptr(), None, ws.data_ptr(),
                                                ws.numel(), stream.cuda_stream))
    threads = [threading.Thread(target=work, args=a) for a in args]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert said == [0] * 200 and kda.device_status() == 0
    for c, a in zip(cases, args):
        c.check(a[3][None], None)


def test_a_cache_grows_forks_and_moves():
    """Extend, append, attend, fork, extend both, compact: as a sequence of its own each."""
    g = torch.Generator().manual_seed(4)
    Hq, Hkv, D, pt = 4, 2, 64, 16
    pool = torch.zeros(1, 24, 2, Hkv, pt, D, dtype=torch.bfloat16, device=DEV)
    table, lengths, refs = torch.full((4, 6), -1, dtype=torch.int32, device=DEV), ints([0] * 4), ints([0] * 24)
    whole = {r: (torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)) for r in range(4)}

    def feed(rows, ns):
        now = lengths.tolist()
        assert all(kda.pages_extend(table, lengths, refs, ints(rows), ints([now[r] + n for r, n in zip(rows, ns)]), page_tokens=pt).tolist())
        q, k, v = (torch.randn(sum(ns), h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        off = [0, *np.cumsum(ns).tolist()]
        kda.pages_append(pool[0], table, lengths, k.to(DEV)[None], v.to(DEV)[None], seqs=ints(rows), cu_seqlens=ints(off))
        out = kda.pages_attention(q.to(DEV)[None], pool[0], table, lengths, scale=0.125, seqs=ints(rows), cu_seqlens=ints(off))[0]
        for j, r in enumerate(rows):
            whole[r] = tuple(torch.cat([old, new[off[j]:off[j + 1]].float()]) for old, new in zip(whole[r], (k, v)))
            n = len(whole[r][0])
            flat = torch.stack(whole[r])[None].permute(0, 1, 3, 2, 4)              # one page of all its tokens
            want, size, _ = ref.attention(q[off[j]:off[j + 1]], flat, torch.tensor([[0]]), torch.tensor([n]), [0], [0, ns[j]], 0.125, 0)
            err = (ref.d(out[off[j]:off[j + 1]]) - want).abs()
            assert bool((err <= (2.0 ** -8 + 1e-4) * size + 2.0 ** -8 * want.abs()).all())

    feed([2, 0], [37, 20])
    feed([0, 2], [1, 1])
    assert kda.pages_fork(pool, table, lengths, refs, ints([2]), ints([3]), page_tokens=pt).tolist() == [1]
    whole[3] = whole[2]
    feed([3, 2], [1, 15])
    kda.pages_free(table, lengths, refs, ints([0]))
    whole[0] = whole[1]
    kda.pages_compact(pool, table, refs)
    feed([2, 3, 0], [1, 1, 5])
    feed([0, 3], [30, 2])
    assert kda.device_status() == 0


@pytest.mark.parametrize("what", ["pool", "heads", "table", "lengths", "seqs", "packed", "expanded", "window", "scale", "overlap", "lse", "kv"])
def test_refusals(what):
    c = Case([50, 60], [3, 3], 4, 2, 64, 16, "bf16", dirty=False)
    q, pool, table, lengths = c.q.to(DEV).view(2, 3, 4, 64), c.pool.to(DEV), c.table.to(DEV), c.lengths.to(DEV)
    kw, err = dict(scale=0.1, seqs=c.seqs.to(DEV)), ValueError
    if what == "pool":
        pool = pool[..., :32].contiguous()
    elif what == "heads":
        q, err = q[:, :, :3].contiguous(), kda.KdaError
    elif what == "table":
        table = table.long()
    elif what == "lengths":
        lengths = lengths[:2]
    elif what == "seqs":
        kw["seqs"] = ints([0])
    elif what == "packed":
        kw["cu_seqlens"] = ints([0, 3, 6])
    elif what == "expanded":
        q = q[:, :1].expand(2, 3, 4, 64)
    elif what == "window":
        kw["window"], err = -1, kda.KdaError
    elif what == "scale":
        kw["scale"], err = float("nan"), kda.KdaError
    elif what == "overlap":
        kw["out"], err = q, kda.KdaError
    elif what == "lse":
        kw["lse"] = torch.zeros(2, 3, 3, device=DEV)
    else:
        k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device=DEV)
        with pytest.raises(ValueError):
            kda.pages_append(pool, table, lengths, k, k[:, :, :1], seqs=c.seqs.to(DEV))
        with pytest.raises(ValueError):
            kda.pages_append(pool, table, lengths, k[:, :, :1], k[:, :, :1], seqs=c.seqs.to(DEV))
        return
    with pytest.raises(err):
        kda.pages_attention(q, pool, table, lengths, **kw)
