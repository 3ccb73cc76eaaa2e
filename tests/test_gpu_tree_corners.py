"""Drafted-token calls at the ends of their ranges: lengths and positions near the largest,
capacities that are passed, values that are not finite, calls directly behind one another."""
import math

import numpy as np
import pytest
import torch

import tree_ref as R
from compressed_sparse_mqa_gb300 import ds4a
from test_gpu_tree import NAN16, Cache, attn_setup, check_attn, comp_setup, dev, no_error, run_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["append", "compress", "attn", "commit"])
@pytest.mark.parametrize("ln", [(1 << 63) - 1, (1 << 63) - 4, 1 << 62])
def test_lengths_near_the_end_of_int64_are_refused(call, ln):
    """len + n does not fit 64 bits: the session is past its pages all the same, and is left alone."""
    rng = np.random.default_rng(1)
    N, ratio, D, H = 4, 2, 64, 8
    c, par, q, _, _, _ = attn_setup(rng, [21, 34, 15], [4, 4, 3], N, H, D, 16, 64, 0, 0, "tree")
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, ratio, D)
    c.lens[1] = ln
    kv = c.upload()
    kn = torch.ones(3, N, D, dtype=torch.float16, device="cuda")
    lo, so = torch.full((3,), -9, device="cuda"), torch.full_like(state, 5.0)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(3, N, H, D), dtype=torch.uint8, device="cuda")
    own = torch.from_numpy(c.rows(1, range(c.mp * c.page))).cuda()       # session 1's pool rows
    mine = lambda: [c.dk.view(-1, D)[own], c.dv.view(-1, D)[own], dck[1], dcv[1], lo[1], so[1], out[1]]
    before = [t.clone() for t in mine()]
    if call == "append":
        ds4a.ds4a_paged_append(kv, kn, kn, c.dn, dev(par))
    elif call == "compress":
        ds4a.ds4a_compress_tree(kv, c.dn, dev(par), dw, ratio, state, dck, dcv)
    elif call == "attn":
        ds4a.ds4a_attn_tree(kv, dev(q), c.dn, dev(par), 64, None, None, 0, None, 0.1, out, ws)
    else:
        leaf = torch.tensor([3, 3, 2], dtype=torch.int32, device="cuda")
        ds4a.ds4a_commit_tree(kv, c.dn, dev(par), leaf, lo, dw, ratio, state, so, dck, dcv)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == ds4a.DS4A_ERR_CAPACITY
    for b, a in zip(before, mine()):
        assert torch.equal(b.view(-1).view(torch.uint8), a.contiguous().view(-1).view(torch.uint8))
    if call == "attn":
        c.n[1] = 0
        check_attn(c, par, q, None, None, None, 64, 0, 0.1, out)
    if call == "commit":
        assert lo.tolist() == [21 + len(R.paths_of(par[0], 4)[3]), -9, 15 + len(R.paths_of(par[2], 3)[2])]


def test_compress_tree_leaves_committed_rows_past_the_capacity_alone():
    """Session 0 has more committed rows than lie before the draft's: those rows keep their bits."""
    rng = np.random.default_rng(8)
    N, D = 4, 64
    c = Cache(rng, [6, 3], [4, 4], D, 16, N)
    c.draft()
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, 1, D)
    keep = 4 + N                                     # rows 0 .. 3 before the draft's; session 0 has six
    dck, dcv = dck[:, :keep].contiguous(), dcv[:, :keep].contiguous()
    before = dck.clone(), dcv.clone()
    ds4a.ds4a_compress_tree(c.upload(), c.dn, None, dw, 1, state, dck, dcv, N=N)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == ds4a.DS4A_ERR_CAPACITY
    for b, a in zip(before, (dck, dcv)):
        assert torch.equal(b[0].view(torch.int16), a[0].view(torch.int16))
        assert torch.isfinite(a[1, 4:]).all()        # session 1's four rows (a row of one token is the token)
    at = c.rows(1, range(3, 7))
    assert np.array_equal(dck[1, 4:].cpu().numpy(), c.k[at]) and np.array_equal(dcv[1, 4:].cpu().numpy(), c.v[at])
