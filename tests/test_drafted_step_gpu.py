"""The drafted step of examples/drafted_step.py against the same tokens taken one by one."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import drafted_step as ex  # noqa: E402

from _parity import assert_states_close  # noqa: E402

pytestmark = pytest.mark.gpu


def test_states_and_cache_advance_as_token_by_token():
    B = 3
    m, one = ex.Model(B, pages_each=4), ex.Model(B, pages_each=4)
    last = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    history = [[] for _ in range(B)]
    for _ in range(5):
        tokens, accepted = ex.step(m, last, ex.DRAFTS)
        for b in range(B):
            row, j = tokens[b].tolist(), int(accepted[b])
            assert all(t >= 0 for t in row[:j + 1]) and all(t == -1 for t in row[j + 1:])
            history[b] += [int(last[b])] + row[:j]
        last = tokens.gather(1, accepted[:, None].long())[:, 0].contiguous()
    assert m.lens.tolist() == [len(h) for h in history]
    # the same tokens, one per call: a request that has run out goes on with its last one
    # on a slot that is not looked at
    for i in range(max(len(h) for h in history)):
        live = torch.tensor([i < len(h) for h in history], device="cuda")
        token = torch.tensor([h[min(i, len(h) - 1)] for h in history], device="cuda")
        x = one.embed[token]
        h = one.kda(x, cu, torch.where(live, one.slots, one.slots + B))
        one.lens += live.to(torch.int32)
        one.attention(h, cu, torch.full_like(one.lens, i + 1), 1)
    assert_states_close(m.pool[:B].cpu().numpy(), one.pool[:B].double().cpu().numpy())
    # the cache: codes of equal rows may differ by the rounding of a window's other shapes of
    # the same products, so the rows are compared as values, within a step of e4m3
    for name in ("k", "v"):
        code, scale = getattr(m, name + "_cache").float(), getattr(m, name + "_scale")
        ref, ref_scale = getattr(one, name + "_cache").float(), getattr(one, name + "_scale")
        for b in range(B):
            for pos in range(len(history[b])):
                at = (int(m.table[b, pos // ex.PAGE]), slice(None), pos % ex.PAGE)
                x, y = code[at] * scale[at][:, None], ref[at] * ref_scale[at][:, None]
                assert bool(((x - y).abs() <= 2.0 ** -3 * y.abs() + 2.0 ** -8 * ref_scale[at][:, None]).all())


def test_main_runs(capsys):
    ex.main()
    assert "lengths" in capsys.readouterr().out
