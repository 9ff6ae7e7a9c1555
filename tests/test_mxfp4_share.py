"""A share of MXFP4 experts as the expert calls see it: its own tokens and their choices.  Without a
GPU: a call whose arguments are all valid reaches the device check."""
import os

import pytest

from test_mxfp4_refusals import DOWN, PACK, UP, P, bad, fine


@pytest.fixture(scope="module")
def L():
    from mixture_experts_layer_added_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_added_amd import build
        build.build(verbose=False)
    return _lib


@pytest.fixture
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the valid call would run")


FEW = dict(E=2, G=1, M=1, J=1, S=0)  # fewer experts than a token has choices


def test_more_choices_than_experts(L, no_gpu):
    lib = L.lib()
    for f, good in ((lib.moe_pack_expert_weights_mxfp4, PACK), (lib.moe_expert_ffn_up_mxfp4, UP),
                    (lib.moe_expert_ffn_down_mxfp4, DOWN)):
        for K in (3, 16):
            fine(L, f, {"p": P(L, K=K, **FEW), **good})


def test_choices_keep_their_limits(L):
    lib = L.lib()
    for f, good in ((lib.moe_pack_expert_weights_mxfp4, PACK), (lib.moe_expert_ffn_up_mxfp4, UP),
                    (lib.moe_expert_ffn_down_mxfp4, DOWN)):
        for K in (0, 17):
            bad(L, f(P(L, K=K, **FEW), *good.values()), "K=")
    # what routes to the experts still needs as many of them
    from test_mxfp4_refusals import A
    p = P(L, K=3, **FEW)
    bad(L, lib.moe_route(p, A, A, A, A, A, A, A, A, 1 << 30, None), "exceeds")
    bad(L, lib.moe_permute(p, A, A, A, A, A, None, None, A, 1 << 30, None), "exceeds")


def test_rows_of_x_are_the_tokens(L, no_gpu):
    """The limit on x is that of its T rows, whatever their choices make of them."""
    big = dict(T=65000, H=65536, I=128, K=16, **FEW)
    fine(L, L.lib().moe_expert_ffn_up_mxfp4, {"p": P(L, **big), **UP, "ldxs": 2048})
    bad(L, L.lib().moe_expert_ffn_up_mxfp4(P(L, **{**big, "T": 65536}), *{**UP, "ldxs": 2048}.values()),
        "2^31")


def test_sort_of_no_tokens_needs_offsets_alone(L, no_gpu):
    from test_mxfp4_refusals import SORT
    none = {**SORT, "T": 0, "idx": None, "tok": None, "row": None, "ws": None, "ws_bytes": 0}
    fine(L, L.lib().moe_sort_by_expert, none)
    bad(L, L.lib().moe_sort_by_expert(*{**none, "off": None}.values()), "offsets")
