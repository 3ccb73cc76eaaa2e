"""Refusals of the drafted-token calls that return before a CUDA call: outputs that overlap inputs in part."""
from test_tree_host import ARG, FAKE, attn, commit, kv


def test_commit_refuses_outputs_that_overlap_their_inputs_in_part(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    state = 2 * (2 + 2 * 128) * 4
    for kw in (dict(lo=FAKE + 8), dict(lo=FAKE - 8), dict(so=FAKE + 4), dict(so=FAKE + state // 2), dict(so=FAKE + state - 4),
               dict(so=FAKE - state + 4)):
        assert commit(L, c, **kw) == ARG, kw


def test_attn_refuses_scales_whose_base_2_form_is_not_finite(ds4a_lib):
    for scale in (2.4e38, 2.9e38, 3.4e38):
        assert attn(ds4a_lib.lib(), kv(ds4a_lib), scale=scale) == ARG
