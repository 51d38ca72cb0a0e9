"""The served decoder: steps on the cache continue prompts, through forks, ended requests and compaction.

The steps' logits are compared with the prompt path's on the whole sequences.  The tolerance is the package's
for bf16 results, 2e-2 of the rms, on states and histories that are the same up to rounding; the four layers and
the products between them carry on what each layer's bf16 rounding (2^-9) leaves, hence three times that."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gated_delta_rule_sm_gb300 as kda  # noqa: E402
from gated_delta_rule_sm_gb300 import serve  # noqa: E402


def ids(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_steps_continue_prompts_through_forks_and_compaction():
    model = serve.Decoder()
    lengths, more = [37, 150, 5], 6
    g = torch.Generator().manual_seed(3)
    seqs = [torch.randint(0, 512, (n + more,), generator=g) for n in lengths]
    extra = torch.cat([seqs[0][:lengths[0]], torch.randint(0, 512, (more,), generator=g)])    # a fork of the first
    whole = [*seqs, extra]
    ref_cache = serve.StateCache(model, slots=4, sequences=4)
    ref_cache.admit(ids(0, 1, 2, 3), ids(*(len(s) for s in whole)))
    cu = serve.offsets([len(s) for s in whole])
    want = serve.prompt(model, ref_cache, torch.cat(whole)[None].cuda(), cu, ids(0, 1, 2, 3))[0]

    cache = serve.StateCache(model, slots=7, sequences=5)
    cache.admit(ids(4, 0, 1, 2), ids(1, *lengths))     # row 4 holds a page that is given up below
    cut = torch.cat([s[:n] for s, n in zip(seqs, lengths)])[None].cuda()
    serve.prompt(model, cache, cut, serve.offsets(lengths), ids(0, 1, 2))
    assert cache.fork(ids(0), ids(3)).tolist() == [1]
    rows = ids(0, 1, 2, 3)
    for k in range(more):
        if k == 3:
            cache.release(ids(4))
            cache.compact()
            assert sorted(cache.slots(rows).tolist()) == [0, 1, 2, 3]
        n = [*lengths, lengths[0]]
        now = torch.stack([s[m + k] for s, m in zip(whole, n)]).cuda()
        got = serve.step(model, cache, now, rows)
        for r in range(4):
            ref = want[int(cu[r]) + n[r] + k]
            err = (got[r] - ref).abs().max() / ref.square().mean().sqrt()
            assert float(err) <= 6e-2, (k, r, float(err))
    for pool, ref_pool in zip(cache.pools, ref_cache.pools):
        a = pool["state"][0][cache.slots(rows).long()]
        b = ref_pool["state"][0][ref_cache.slots(rows).long()]
        assert float((a - b).norm() / b.norm()) <= 6e-2
    assert kda.device_status() == 0


def test_command_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["serve", "--prompts", "9", "70", "--samples", "2", "--steps", "3", "--layers", "2"])
    serve.main()
    assert "us a step" in capsys.readouterr().out
