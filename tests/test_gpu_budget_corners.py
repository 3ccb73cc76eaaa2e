"""Calls on caches held to a budget that the other tests do not make."""
import numpy as np
import pytest
import torch

import budget_ref as E
from compressed_sparse_mqa_gb300 import ds4a
from test_gpu_budget import last_error
from test_gpu_tree import Cache, dev

pytestmark = pytest.mark.gpu


# ---- eviction ----------------------------------------------------------------------------------

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ln,other,budget,bad", [
    (30, 80, 40, 1),                # one CTA a session
    (3000, 3500, 3200, 187),        # a cluster: its last page
    (600 * 16, 9700, 9650, 514),    # more pages than a CTA has threads
])
def test_evict_uncut_session_with_a_bad_page_is_left_alone(ln, other, budget, bad, in_place):
    """A page id outside the pool among a session's tokens leaves it alone, whether it would be cut or not; a bad entry
    behind them does not matter."""
    rng = np.random.default_rng(ln)
    c = Cache(rng, [ln, other, ln], [0] * 3, 64, 16, 16)
    c.table[0, bad] = c.n_pages
    c.table[2, (ln - 1) // 16 + 1] = -1
    kv = c.upload()
    S = c.mp * 16
    acc, pos = rng.random((3, S)).astype(np.float32), np.tile(np.arange(S, dtype=np.int32), (3, 1))
    da, dp = dev(acc), dev(pos)
    ao, po = (da, dp) if in_place else (torch.full_like(da, 5), torch.full_like(dp, 6))
    lo = torch.full_like(c.dlen, -4)
    ws = torch.zeros(ds4a.ds4a_evict_workspace_bytes(3, S, budget), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_evict(kv, da, dp, torch.tensor([ln, other, ln], device="cuda"), budget, 2, 5, ao, po, lo, ws)
    assert last_error() == 7
    assert lo.tolist() == [-4, budget, ln]
    want_a, want_p = (acc[0], pos[0]) if in_place else (np.full(S, 5, np.float32), np.full(S, 6, np.int32))
    assert np.array_equal(ao[0].cpu().numpy(), want_a) and np.array_equal(po[0].cpu().numpy(), want_p)
    assert np.array_equal(ao[2, :ln].cpu().numpy(), acc[2, :ln])
    place, _ = E.evict(acc[1], pos[1], other, other, budget, 2, 5)
    assert np.array_equal(po[1, :budget].cpu().numpy(), pos[1, place])
