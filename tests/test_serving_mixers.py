"""The served decoder with gated recurrences and attention among its layers: steps and further chunks on the caches
continue prompts, through forks, ended requests and compaction.

The logits are compared with the prompt path's on the whole sequences, with the tolerance of the example's other test: the
package's 2e-2 of the rms for bf16 results, three times that for four layers and the products between them."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_delta_rule_sm_gb300 as kda  # noqa: E402
from gated_delta_rule_sm_gb300 import serve  # noqa: E402

TOL = 6e-2


def ids(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def close(got, want):
    return float((got - want).abs().max() / want.square().mean().sqrt()) <= TOL


@pytest.mark.parametrize("pattern", ["dsga", "ag", "gads"])
def test_steps_and_chunks_continue_prompts(pattern):
    model = serve.Decoder(pattern=pattern)
    lengths, chunk, more = [37, 150, 5], [20, 3, 40], 5
    g = torch.Generator().manual_seed(3)
    seqs = [torch.randint(0, 512, (n + c + more,), generator=g) for n, c in zip(lengths, chunk)]
    first = lengths[0] + chunk[0]
    extra = torch.cat([seqs[0][:first], torch.randint(0, 512, (more,), generator=g)])    # a fork of the first
    whole = [*seqs, extra]
    ref_cache = serve.StateCache(model, slots=4, sequences=4)
    assert ref_cache.admit(ids(0, 1, 2, 3), ids(*(len(s) for s in whole))).tolist() == [1] * 4
    cu = serve.offsets([len(s) for s in whole])
    want = serve.prompt(model, ref_cache, torch.cat(whole)[None].cuda(), cu, ids(0, 1, 2, 3))[0]

    cache = serve.StateCache(model, slots=7, sequences=5)
    cache.admit(ids(4, 0, 1, 2), ids(33, *lengths))     # row 4 holds pages that are given up below
    cut = torch.cat([s[:n] for s, n in zip(seqs, lengths)])[None].cuda()
    serve.prompt(model, cache, cut, serve.offsets(lengths), ids(0, 1, 2))
    # a second chunk of each prompt
    assert cache.grow(ids(0, 1, 2), ids(*chunk)).tolist() == [1] * 3
    cut = torch.cat([s[n:n + c] for s, n, c in zip(seqs, lengths, chunk)])[None].cuda()
    off = serve.offsets(chunk)
    got = serve.prompt(model, cache, cut, off, ids(0, 1, 2), more=True)[0]
    for r in range(3):
        a = int(cu[r]) + lengths[r]
        assert close(got[int(off[r]):int(off[r + 1])], want[a:a + chunk[r]]), r
    assert cache.fork(ids(0), ids(3)).tolist() == [1]
    rows, n = ids(0, 1, 2, 3), [a + b for a, b in zip(lengths, chunk)] + [first]
    for k in range(more):
        if k == 3:
            cache.release(ids(4))
            cache.compact()
            assert sorted(cache.slots(rows).tolist()) == [0, 1, 2, 3]
            held = cache.kv_table[cache.kv_table >= 0]
            assert cache.kv is None or int(held.max()) == int((cache.kv_refs > 0).sum()) - 1
        now = torch.stack([s[m + k] for s, m in zip(whole, n)]).cuda()
        got = serve.step(model, cache, now, rows)
        for r in range(4):
            assert close(got[r], want[int(cu[r]) + n[r] + k]), (k, r)
    assert kda.device_status() == 0


def test_refused_admissions_and_forks_leave_no_pages():
    """Where one of the two caches is full, the other gives its page back."""
    model = serve.Decoder(layers=2, pattern="ga")
    cache = serve.StateCache(model, slots=4, sequences=5, kv_pages=4, kv_row=4)
    assert cache.admit(ids(0, 1), ids(40, 40)).tolist() == [1, 0]           # 3 of 4 pages, then 3 more
    assert cache.lengths.tolist()[:2] == [40, 0] and int((cache.refs > 0).sum()) == 1
    assert cache.admit(ids(2), ids(9)).tolist() == [1]
    assert cache.fork(ids(0), ids(3)).tolist() == [0]                       # its last page would need a fifth
    assert int((cache.refs > 0).sum()) == 2 and int(cache.kv_lengths[3]) == 0
    cache.release(ids(2))
    assert cache.fork(ids(0), ids(3)).tolist() == [1]
    assert sorted(cache.kv_refs.tolist()) == [1, 1, 2, 2]
    assert kda.device_status() == 0


def test_a_longer_admission_that_is_refused_changes_nothing():
    """A row that holds its states and keys already keeps them where there is no room for more, and goes on."""
    model = serve.Decoder(pattern="dsga")
    g = torch.Generator().manual_seed(6)
    prompts, nxt = torch.randint(0, 512, (1, 50), generator=g).cuda(), torch.randint(0, 512, (2, 3), generator=g).cuda()
    rows, off = ids(0, 1), serve.offsets([20, 30])
    caches = [serve.StateCache(model, slots=4, sequences=3, kv_pages=n, kv_row=6) for n in (18, 5)]
    for cache in caches:
        assert cache.admit(rows, ids(20, 30)).tolist() == [1] * 2                     # 2 pages each
        serve.prompt(model, cache, prompts, off, rows)
    plenty, few = caches
    held = few.table.clone(), few.kv_table.clone()
    assert few.admit(ids(1, 2, 0), ids(90, 40, 60)).tolist() == [0] * 3               # 6, 3 and 4 pages of keys: one is free
    assert torch.equal(few.table, held[0]) and torch.equal(few.kv_table, held[1])
    assert few.lengths.tolist() == [20, 30, 0] and few.kv_lengths.tolist() == [20, 30, 0]
    assert int((few.refs > 0).sum()) == 2 and int((few.kv_refs > 0).sum()) == 4
    for k in range(2):
        want, got = (serve.step(model, cache, nxt[:, k], rows) for cache in caches)
        assert all(close(got[r], want[r]) for r in range(2))
    assert few.admit(ids(1), ids(40)).tolist() == [1] and few.lengths.tolist() == [20, 40, 0]
    assert few.admit(ids(-1, 3, 99), ids(5, 5, 5)).tolist() == [0] * 3                # rows that are none
    assert few.lengths.tolist() == [20, 40, 0] and few.kv_lengths.tolist() == [22, 40, 0]
    assert kda.device_status() == 0


def test_a_step_without_a_free_page_changes_nothing():
    """Its row is left as it was, gets NaN, and goes on when there is a page again; the other rows do not notice."""
    model = serve.Decoder(pattern="dsga")
    g = torch.Generator().manual_seed(5)
    prompts, nxt = torch.randint(0, 512, (1, 62), generator=g).cuda(), torch.randint(0, 512, (2, 3), generator=g).cuda()
    rows, off = ids(0, 1), serve.offsets([30, 32])
    caches = [serve.StateCache(model, slots=4, sequences=3, kv_pages=n, kv_row=4) for n in (12, 5)]
    for cache in caches:
        assert cache.admit(ids(0, 1, 2), ids(30, 32, 9)).tolist() == [1] * 3      # 2, 2 and 1 pages
        serve.prompt(model, cache, prompts, off, rows)
    plenty, few = caches
    want = [serve.step(model, plenty, nxt[:, k], rows) for k in range(3)]
    for k in range(2):
        got = serve.step(model, few, nxt[:, k], rows)                             # row 1 would need a third page
        assert close(got[0], want[k][0]) and bool(torch.isnan(got[1]).all())
    assert few.kv_lengths.tolist() == [32, 32, 9]
    few.release(ids(2))
    for k in range(3):
        assert close(serve.step(model, few, nxt[1:, k], rows[1:])[0], want[k][1])
    assert kda.device_status() == 0


def test_command_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["serve", "--prompts", "9", "70", "--samples", "2", "--steps", "3", "--layers", "4", "--pattern", "dgas"])
    serve.main()
    assert "us a step" in capsys.readouterr().out


@pytest.mark.parametrize("pattern", ["", "aa", "dx"])
def test_patterns_that_are_none(pattern):
    with pytest.raises(ValueError):
        serve.Decoder(pattern=pattern)
