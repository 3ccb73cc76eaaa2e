"""TreeDecodeLayer against DecodeLayer: every node of a checked draft gives what decoding its
path token by token gives, and accepted paths leave the layer where those steps leave it."""
import dataclasses

import numpy as np
import pytest
import torch

import tree_ref as R
from compressed_sparse_mqa_gb300 import configs, ds4a, synth
from compressed_sparse_mqa_gb300.layer import DecodeLayer, TreeDecodeLayer

pytestmark = pytest.mark.gpu


def instances(layer, positions, H=64, D=128, W=128, d_idx=128):
    ratio, topk = {0: (0, 0), 2: (4, 512), 3: (128, 0), 5: (4, 20)}[layer]
    insts = [synth.decode_instance(seed=40 + s, layer=layer, H=H, D=D, window=W, ratio=ratio, d_idx=d_idx, topk=topk, p=p,
                                   sigma_w=configs.SIGMA_W) for s, p in enumerate(positions)]
    return [dataclasses.replace(i, w=insts[0].w) for i in insts]


def gather_h(t):
    return t.detach().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("layer,positions", [(0, [300, 5]), (2, [3001, 402, 6]), (3, [1270, 126, 900]), (5, [515, 30])])
def test_checked_drafts_equal_stepwise_decode(layer, positions):
    insts = instances(layer, positions)
    B, N, H, D, DI = len(insts), 9, 64, 128, 128
    T = TreeDecodeLayer(insts, max_nodes=N, room=64, page=16)
    singles = []
    for inst in insts:
        L = DecodeLayer(inst, cap_extra=40)
        L.step()
        singles.append(L)
    rng = np.random.default_rng(layer)
    rnd = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda()
    for turn in range(3):
        k, v, q, qi, ki = rnd(B, N, D), rnd(B, N, D), rnd(B, N, H, D), rnd(B, N, DI), rnd(B, N, DI)
        par = R.random_parents(rng, B, N)
        n = [N - s for s in range(B)]
        out = T.verify(k, v, q, par, n, qi if T.topk else None, ki if T.topk else None).clone()
        torch.cuda.synchronize()
        assert ds4a.ds4a_last_device_error() == 0
        leaf = [int(rng.integers(0, n[s])) for s in range(B)]
        for s in range(B):
            paths = R.paths_of(par[s], n[s])
            after = None
            for i, path in enumerate(paths):
                C = singles[s].clone()
                C.ring_k, C.ring_v = C.ring_k.clone(), C.ring_v.clone()
                for j in path:
                    ref = C.advance(k[s, j], v[s, j], q[s, j], qi[s, j] if C.topk else None, ki[s, j] if C.topk else None)
                torch.cuda.synchronize()
                if T.topk:
                    assert T.sel[s, i].tolist() == C.sel.tolist(), (s, i)      # the same rows are kept
                # two 16-bit results of one value, both within the repository's 2e-3 of it
                assert float((ref.float() - out[s, i].float()).abs().max()) <= 4e-3, (turn, s, i)
                if i == leaf[s]:
                    after = C
            singles[s] = after
        T.accept(leaf)
        torch.cuda.synchronize()
        assert ds4a.ds4a_last_device_error() == 0
        for s, C in enumerate(singles):
            assert T.len_host[s] == C.p + 1 == int(T.length[s])
            if T.ratio:
                m = (C.p + 1) // T.ratio
                assert torch.equal(T.comp_k[s, :m], C.comp_k[:m]) and torch.equal(T.comp_v[s, :m], C.comp_v[:m])
                if (C.p + 1) % T.ratio:
                    assert torch.equal(T.state[s], C.state)
                if T.topk:
                    assert torch.equal(T.kidx[s, :m], C.kidx[:m])


def test_rotation_on_the_way_in():
    """A layer with rope gives what one without gives on keys and queries rotated beforehand."""
    insts = instances(0, [200, 70])
    inv = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    A = TreeDecodeLayer(insts, max_nodes=5, room=32, rope=(inv, 64, True))
    Bl = TreeDecodeLayer(insts, max_nodes=5, room=32)
    rng = np.random.default_rng(0)
    k, v, q = (torch.from_numpy(rng.standard_normal(s).astype(np.float16)).cuda() for s in ((2, 5, 128), (2, 5, 128), (2, 5, 64, 128)))
    par, n = [[-1, 0, 0, 1, 2]] * 2, [5, 3]
    out = A.verify(k, v, q, par, n).clone()
    kr, qr = k.clone(), q.clone()
    for s in range(2):
        for i, path in enumerate(R.paths_of(np.array(par[s]), n[s])):
            pos = A.len_host[s] + len(path) - 1
            for t in (kr[s, i], qr[s, i]):
                t.copy_(torch.from_numpy(R.rotate(gather_h(t), pos, inv.cpu().numpy(), 64, True).astype(np.float16)))
    ref = Bl.verify(kr, v, qr, par, n)
    torch.cuda.synchronize()
    for s in range(2):   # rotations that round the other way: one step of 2^-10 in a key or query value here and there
        assert float((out[s, :n[s]].float() - ref[s, :n[s]].float()).abs().max()) <= 4e-3


def test_layer_refuses_bad_drafts():
    T = TreeDecodeLayer(instances(2, [100]), max_nodes=4, room=6)
    k, q, qi = torch.zeros(1, 4, 128).half().cuda(), torch.zeros(1, 4, 64, 128).half().cuda(), torch.zeros(1, 4, 128).half().cuda()
    with pytest.raises(ValueError, match="earlier node"):
        T.verify(k, k, q, [[-1, 1, 0, 0]], [4], qi, qi)
    with pytest.raises(ValueError, match="earlier node"):
        T.verify(k, k, q, [[-1, 0, 0, 0]], [5], qi, qi)
    with pytest.raises(ValueError, match="indexer queries"):
        T.verify(k, k, q, [[-1, 0, 0, 0]], [4])
    T.verify(k, k, q, [[-1, 0, 1, 2]], [4], qi, qi)
    with pytest.raises(ValueError, match="accept"):
        T.accept([4])
    T.accept([3])
    with pytest.raises(ValueError, match="no room"):
        T.verify(k, k, q, [[-1, 0, 1, 2]], [4], qi, qi)
    with pytest.raises(ValueError, match="accept"):   # the draft was used up
        T.accept([0])
    with pytest.raises(ValueError, match="nodes"):
        TreeDecodeLayer(instances(0, [100]), max_nodes=65)
