"""TreeDecodeLayer when a call on it fails, and when the caller's arrays change after one."""
import dataclasses

import numpy as np
import pytest
import torch

from compressed_sparse_mqa_gb300 import ds4a
from compressed_sparse_mqa_gb300.layer import TreeDecodeLayer
from test_gpu_tree_layer import instances

pytestmark = pytest.mark.gpu

N = 5


def draft(seed, parent, n=N):
    """One session's draft: verify's arguments."""
    rng = np.random.default_rng(seed)
    rnd = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda()
    return dict(k=rnd(1, N, 128), v=rnd(1, N, 128), q=rnd(1, N, 64, 128), parent=np.array([parent], np.int32), n_node=[n],
                q_idx=rnd(1, N, 128), kidx=rnd(1, N, 128))


def state_of(T):
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == 0
    n = T.len_host[0]
    assert T.length.tolist() == [n]
    tok = T.pool_k.view(-1, 128)[:n], T.pool_v.view(-1, 128)[:n]       # one session: its pages in order
    return [t.clone() for t in tok + (T.comp_k[0, :n // 4], T.comp_v[0, :n // 4], T.kidx[0, :n // 4], T.state[0])]


def make():
    return TreeDecodeLayer(instances(2, [100]), max_nodes=N, room=32, page=16)


BAD = {
    "k shape": lambda d: dict(d, k=d["k"][:, :4]), "v shape": lambda d: dict(d, v=d["v"][..., :64]),
    "q shape": lambda d: dict(d, q=d["q"][:, :, :8]), "k type": lambda d: dict(d, k=d["k"].float()),
    "q on the host": lambda d: dict(d, q=d["q"].cpu()), "q layout": lambda d: dict(d, q=d["q"].transpose(1, 2).contiguous().transpose(1, 2)),
    "q_idx shape": lambda d: dict(d, q_idx=d["q_idx"][:, :3]), "q_idx type": lambda d: dict(d, q_idx=d["q_idx"].float()),
    "kidx shape": lambda d: dict(d, kidx=d["kidx"][:, :1]),
    "k missing": lambda d: dict(d, k=None), "kidx missing": lambda d: dict(d, kidx=None), "parent": lambda d: dict(d, parent=[[-1, 0, 2, 0, 0]]),
    "nodes": lambda d: dict(d, n_node=[N + 1]),
}


@pytest.mark.parametrize("what", list(BAD))
def test_a_refused_draft_changes_nothing(what):
    """verify raises before anything changes: the draft before it can still be accepted, as without the
    refused call, and without one there is nothing to accept."""
    T, C = make(), make()
    second = draft(2, [-1, -1, -1, 0, 3])
    with pytest.raises((ValueError, TypeError, ds4a.Ds4aError)):
        T.verify(**BAD[what](second))
    with pytest.raises(ValueError, match="accept"):
        T.accept([0])
    for L in (T, C):
        out = L.verify(**draft(1, [-1, 0, 1, 2, 3])).clone()
    with pytest.raises((ValueError, TypeError, ds4a.Ds4aError)):
        T.verify(**BAD[what](second))
    assert torch.equal(T.out, out)
    T.accept([4])
    C.accept([4])
    for a, b in zip(state_of(T), state_of(C)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("call", ["ds4a_paged_append", "ds4a_compress_tree", "ds4a_indexer_topk", "ds4a_attn_tree"])
def test_a_draft_whose_calls_fail_cannot_be_accepted(call, monkeypatch):
    T, C = make(), make()
    T.verify(**draft(1, [-1, 0, 1, 2, 3]))

    def fails(*a, **kw):
        raise ds4a.Ds4aError(ds4a.DS4A_ERR_CUDA, call)
    with monkeypatch.context() as m:
        m.setattr(ds4a, call, fails)
        with pytest.raises(ds4a.Ds4aError):
            T.verify(**draft(2, [-1, 0, 0, 1, 1]))
    with pytest.raises(ValueError, match="accept"):   # neither draft: the first one's tokens may be overwritten
        T.accept([0])
    T.accept([-1])
    again = draft(3, [-1, 0, 0, 2, 1])
    for L in (T, C):
        L.verify(**again)
        L.accept([3])
    for a, b in zip(state_of(T), state_of(C)):
        assert torch.equal(a, b)


def test_parents_are_the_layers_own_copy():
    """The caller's array of parents may be used again between verify and accept."""
    T, C = make(), make()
    d = draft(1, [-1, 0, 1, 2, 3])
    C.verify(**draft(1, [-1, 0, 1, 2, 3]))
    T.verify(**d)
    d["parent"][:] = -1
    T.accept([4])
    C.accept([4])
    assert T.len_host == C.len_host == [101 + 5]
    for a, b in zip(state_of(T), state_of(C)):
        assert torch.equal(a, b)


def test_layers_that_pool_their_indexer_keys_are_refused_by_name():
    inst = instances(2, [100])[0]
    inst = dataclasses.replace(inst, kidx_tok=np.zeros((inst.raw_k.shape[0], 128), np.float16))
    with pytest.raises(ValueError, match="pool their indexer keys"):
        TreeDecodeLayer([inst], max_nodes=N, room=32, page=16)
