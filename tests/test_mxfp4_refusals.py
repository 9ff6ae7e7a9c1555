"""What the MXFP4 calls and the calls for a share of the experts refuse, without a GPU: every call
below returns its documented status before it touches the device.  A call whose arguments are all
valid reaches the device check, so on a machine without an MI355X it returns MOE_ERR_UNSUPPORTED or
MOE_ERR_HIP, never a refusal."""
import ctypes
import os

import pytest

A, B, C, D, E, F, G = (ctypes.c_void_p(4096 * i) for i in range(1, 8))
ODD = ctypes.c_void_p(4104)
ODDEST = ctypes.c_void_p(4097)
GOOD = dict(T=256, H=256, E=16, G=4, M=2, K=4, J=2, I=128, S=1, act_dtype=1, expert_dtype=3)


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


def P(L, **kw):
    return ctypes.byref(L.problem(**{**GOOD, **kw}))


def bad(L, rc, frag, status=None):
    assert rc == (L.MOE_ERR_INVALID_ARG if status is None else status)
    assert frag in L.last_error(), L.last_error()


def each(L, f, good, wrongs):
    """f with one argument replaced at a time: (name, value, part of the message)."""
    for name, value, frag in wrongs:
        assert name in good
        bad(L, f(*{**good, name: value}.values()), frag)


def fine(L, f, good):
    assert f(*good.values()) in (L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_HIP), L.last_error()


QUANT = dict(x=A, dtype=1, rows=40, cols=100, ldx=100, q=B, ldq=64, scale=C, lds=16, qt=D, ldqt=32,
             st=E, ldst=16, random=F, stream=None)


def test_quantize(L):
    f = L.lib().moe_quantize_mxfp4
    each(L, f, QUANT, [
        ("x", None, "x is NULL"), ("x", ODDEST, "aligned"), ("dtype", 2, "dtype"),
        ("dtype", 3, "dtype"), ("rows", 0, "rows"), ("cols", -1, "cols"), ("rows", 1 << 41, "rows"),
        ("ldx", 99, "ldx"), ("q", ODD, "16-byte"), ("ldq", 48, "row stride"), ("ldq", 72, "row"),
        ("scale", None, "scales"), ("scale", ODD, "scales"), ("lds", 8, "scales"), ("lds", 0, "scal"),
        ("qt", ODD, "16-byte"), ("ldqt", 16, "row stride"), ("st", None, "scales"),
        ("ldst", 4, "scales"), ("q", A, "their own"), ("qt", A, "their own"), ("qt", B, "their own"),
        ("scale", B, "their own"), ("st", C, "their own"), ("q", F, "their own"),
        ("st", F, "their own")])
    none = {**QUANT, "q": None, "qt": None}
    bad(L, f(*none.values()), "both NULL")
    big = {**QUANT, "rows": 128 << 20, "cols": 128 << 3, "ldx": 128 << 3, "ldq": 512, "lds": 32,
           "ldqt": 64 << 20, "ldst": 4 << 20}
    bad(L, f(*big.values()), "blocks")


def test_valid_calls_reach_the_device(L, no_gpu):
    lib = L.lib()
    fine(L, lib.moe_quantize_mxfp4, QUANT)
    fine(L, lib.moe_quantize_mxfp4, {**QUANT, "qt": None, "st": None, "ldqt": 0, "ldst": 0,
                                     "random": None})
    fine(L, lib.moe_dequantize_mxfp4, VALUES)
    fine(L, lib.moe_gemm_mxfp4, PRODUCT)
    for good, f in ((PACK, lib.moe_pack_expert_weights_mxfp4), (UP, lib.moe_expert_ffn_up_mxfp4),
                    (DOWN, lib.moe_expert_ffn_down_mxfp4)):
        fine(L, f, {"p": P(L), **good})
    fine(L, lib.moe_sort_by_expert, SORT)
    for name, good in MOVES.items():
        fine(L, getattr(lib, name), good)
    for name, good in MOVES.items():  # no tokens: no pointers
        empty = {k: None if isinstance(v, ctypes.c_void_p) else v for k, v in good.items()}
        fine(L, getattr(lib, name), {**empty, "T": 0})


VALUES = dict(rows=40, cols=100, q=B, ldq=64, scale=C, lds=16, out=A, ldo=100, dtype=0, stream=None)


def test_values(L):
    each(L, L.lib().moe_dequantize_mxfp4, VALUES, [
        ("rows", 0, "rows"), ("cols", 0, "cols"), ("q", None, "q is NULL"), ("q", ODD, "16-byte"),
        ("ldq", 60, "row stride"), ("scale", None, "scales"), ("lds", 20, "scales"),
        ("out", None, "out is NULL"), ("out", ctypes.c_void_p(4098), "aligned"), ("ldo", 99, "ldo"),
        ("dtype", 3, "dtype"), ("out", B, "its own"), ("out", C, "its own")])


PRODUCT = dict(M=40, N=50, K=100, a=A, lda=64, sa=B, ldsa=16, b=C, ldb=64, sb=D, ldsb=16, c=E, ldc=50,
               c_dtype=0, accumulate=1, ws=F, ws_bytes=1 << 24, stream=None)


def test_product(L):
    f = L.lib().moe_gemm_mxfp4
    each(L, f, PRODUCT, [
        ("M", 0, "M, N"), ("N", 0, "M, N"), ("K", 0, "M, N"), ("M", (1 << 26) + 1, "M, N"),
        ("K", (1 << 22) + 1, "K in"), ("a", None, "a is NULL"), ("a", ODD, "a is not"),
        ("b", None, "b is NULL"), ("c", None, "c is NULL"), ("c", ODD, "c is not"),
        ("lda", 48, "a needs"), ("ldb", 40, "b needs"), ("sa", None, "a's scales"),
        ("sa", ODD, "a's scales"), ("sb", None, "b's scales"), ("ldsa", 4, "a's scales"),
        ("ldsb", 24, "b's scales"), ("lda", 1 << 23, "2^22"), ("ldsb", 1 << 23, "2^22"),
        ("ldc", 49, "ldc"), ("c_dtype", 3, "c_dtype"), ("accumulate", 2, "accumulate"),
        ("c", A, "over an operand"), ("c", C, "over an operand"), ("c", B, "over an operand"),
        ("c", D, "over an operand")])
    bad(L, f(*{**PRODUCT, "c_dtype": 1}.values()), "accumulate")
    big = {**PRODUCT, "M": 1 << 20, "N": 1 << 20, "ldc": 1 << 20}
    bad(L, f(*big.values()), "M*N")
    need = L.moe_gemm_mxfp4_workspace_bytes(64, 64, 16384)
    assert need > 0  # few tiles and many steps: split over k
    split = {**PRODUCT, "M": 64, "N": 64, "ldc": 64, "K": 16384, "lda": 8192, "ldb": 8192,
             "ldsa": 512, "ldsb": 512}
    for ws, n in ((F, need - 1), (None, need), (ODD, need)):
        bad(L, f(*{**split, "ws": ws, "ws_bytes": n}.values()), "workspace", L.MOE_ERR_WORKSPACE)
    assert L.moe_gemm_mxfp4_workspace_bytes(1, 7168, 2048) == 0


PACK = dict(w13=A, s13=B, w2=C, s2=D, p13=E, p2=F, stream=None)
UP = dict(xq=A, xs=B, ldxs=16, tok=C, off=D, w=E, hq=F, hs=G, ldhs=16, stream=None)
DOWN = dict(hq=A, hs=B, ldhs=16, off=C, w=D, y=E, stream=None)


def test_experts(L):
    lib = L.lib()

    def wrong(f, good, wrongs):
        each(L, f, {"p": P(L), **good}, wrongs)
        for kw in (dict(expert_dtype=1), dict(expert_dtype=2)):
            bad(L, f(P(L, **kw), *good.values()), "MXFP4")
        bad(L, f(None, *good.values()), "problem")
        bad(L, f(P(L, act_dtype=0), *good.values()), "dtypes")

    wrong(lib.moe_pack_expert_weights_mxfp4, PACK, [
        ("w13", None, "w13 is NULL"), ("s13", ODD, "w13_scale is not"), ("w2", None, "w2 is NULL"),
        ("s2", None, "w2_scale is NULL"), ("p13", ODD, "aligned"), ("p13", A, "their own"),
        ("p2", D, "their own"), ("p2", E, "their own")])
    bad(L, lib.moe_pack_expert_weights_mxfp4(P(L), A, B, C, D, None, None, None), "both NULL")
    wrong(lib.moe_expert_ffn_up_mxfp4, UP, [
        ("xq", None, "x_q is NULL"), ("xq", ODD, "aligned"), ("xs", None, "x_q's scales"),
        ("ldxs", 4, "x_q's scales"), ("tok", None, "sorted_token"), ("off", None, "offsets"),
        ("w", None, "w13_packed"), ("hq", None, "h_q is NULL"), ("hs", None, "h_q's scales"),
        ("ldhs", 12, "h_q's scales"), ("hq", A, "their own"), ("hs", B, "their own"),
        ("ldxs", 1 << 24, "2^31"), ("ldhs", 1 << 23, "2^22")])
    bad(L, lib.moe_expert_ffn_up_mxfp4(P(L, T=1 << 24), *UP.values()), "2^31")
    for f, good in ((lib.moe_expert_ffn_up_mxfp4, {**UP, "ldxs": 32}),
                    (lib.moe_expert_ffn_down_mxfp4, DOWN)):
        bad(L, f(P(L, T=1 << 26, K=16, M=4, H=128), *good.values()), "2^23")
    wrong(lib.moe_expert_ffn_down_mxfp4, DOWN, [
        ("hq", None, "h_q is NULL"), ("hs", ODD, "h_q's scales"), ("ldhs", 0, "h_q's scales"),
        ("off", None, "offsets"), ("w", None, "w2_packed"), ("y", None, "y_sorted"),
        ("y", A, "its own"), ("ldhs", 1 << 23, "2^22")])
    assert L.moe_mxfp4_packed_bytes(3, 256, 128) == 3 * 256 * 128 * 17 // 32
    for a in ((0, 256, 128), (1, 100, 128), (1, 256, 100), (1, 0, 128)):
        with pytest.raises(L.MoeError):
            L.moe_mxfp4_packed_bytes(*a)


def test_other_calls_refuse_mxfp4_experts(L):
    lib = L.lib()
    U, p = L.MOE_ERR_UNSUPPORTED, P(L)
    bad(L, lib.moe_permute(p, A, A, A, A, A, A, A, A, 1 << 30, None), "x_sorted", U)
    bad(L, lib.moe_permute_noalloc(p, A, A, A, A, A, A, A, None), "x_sorted", U)
    bad(L, lib.moe_expert_ffn(p, A, A, A, A, A, A, A, A, A, 1 << 30, None), "MXFP4", U)
    bad(L, lib.moe_expert_ffn_up(p, A, A, A, A, A, A, A, None), "MXFP4", U)
    bad(L, lib.moe_expert_ffn_up_gather(p, A, A, A, A, A, A, A, A, None), "MXFP4", U)
    bad(L, lib.moe_expert_ffn_down(p, A, A, A, A, A, A, None), "MXFP4", U)
    assert L.moe_workspace_bytes(L.problem(**GOOD), L.MOE_CALL_EXPERT_FFN) == 0
    assert "MXFP4" in L.last_error()
    bad(L, lib.moe_combine_backward(p, A, A, A, A, A, A, None), "backward", U)
    bad(L, lib.moe_router_backward(p, *[A] * 11, None), "backward", U)
    bad(L, lib.moe_unpermute_sum(p, A, A, A, A, None), "backward", U)
    bad(L, lib.moe_expert_ffn_up_save(p, A, A, A, A, A, A, None), "backward", U)
    bad(L, lib.moe_expert_ffn_backward_input(p, *[A] * 7, None), "backward", U)
    bad(L, lib.moe_expert_ffn_backward_weight(p, *[A] * 8, None), "backward", U)
    bad(L, lib.moe_checkpoint_save(p, A, B, C, None), "backward", U)
    bad(L, lib.moe_checkpoint_restore(p, A, B, C, D, None), "backward", U)
    for f, n in ((lib.moe_pack_expert_weights, 4), (lib.moe_pack_expert_weights_transposed, 4),
                 (lib.moe_expert_ffn_up_packed, 10), (lib.moe_expert_ffn_down_packed, 6),
                 (lib.moe_expert_ffn_backward_input_packed, 7),
                 (lib.moe_expert_ffn_backward_input_checkpoint, 9)):
        rc = f(p, *[ctypes.c_void_p(4096 * (i + 1)) for i in range(n)], None)
        assert rc in (L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_INVALID_ARG), f
        assert "not gfx950" not in L.last_error()  # refused before the device is looked at


SORT = dict(T=300, K=8, idx=A, first=3, count=20, off=B, tok=C, row=D, ws=E, ws_bytes=1 << 20,
            stream=None)


def test_sort(L):
    f = L.lib().moe_sort_by_expert
    each(L, f, SORT, [
        ("T", -1, "T="), ("T", 1 << 29, "T="), ("K", 0, "K="), ("K", 17, "K="), ("count", 0, "count"),
        ("count", 513, "count"), ("first", -1, "first"), ("idx", None, "topk_idx"),
        ("off", None, "offsets"), ("tok", None, "sorted_token"), ("row", None, "pair_row"),
        ("row", A, "their own"), ("tok", A, "their own"), ("tok", D, "their own")])
    need = L.moe_sort_by_expert_workspace_bytes(300, 8, 20)
    assert need == (3 + 1) * 20 * 4 + 16
    for ws, n in ((E, need - 1), (None, need), (ODD, need)):
        bad(L, f(*{**SORT, "ws": ws, "ws_bytes": n}.values()), "workspace", L.MOE_ERR_WORKSPACE)
    for a in ((-1, 8, 20), (300, 0, 20), (300, 8, 513)):
        with pytest.raises(L.MoeError):
            L.moe_sort_by_expert_workspace_bytes(*a)


_ONE = dict(dtype=1, T=30, K=4, H=100, x=A, ldx=100, row=B, w=C, o=D, ldo=100, stream=None)
_TWO = dict(dtype=1, T=30, K=4, H=100, x=A, ldx=100, row=B, w=C, y=E, ldy=100, o=D, ldo=100, dw=F,
            stream=None)
MOVES = dict(moe_dispatch=_ONE, moe_collect=_ONE, moe_dispatch_backward=_TWO,
             moe_collect_backward=_TWO)


@pytest.mark.parametrize("name", MOVES)
def test_moves(L, name):
    f, good = getattr(L.lib(), name), MOVES[name]
    each(L, f, good, [
        ("dtype", 2, "dtype"), ("T", -1, "T="), ("K", 17, "K="), ("H", 0, "H="),
        ("H", (1 << 20) + 1, "H="), ("x", None, "is NULL"), ("x", ODDEST, "aligned"),
        ("ldx", 99, "row stride"), ("ldx", 1 << 32, "row stride"), ("row", None, "pair_row"),
        ("o", None, "is NULL"), ("o", ODDEST, "aligned"), ("ldo", 99, "row stride"),
        ("o", A, "its own")])
    if good is _TWO:
        each(L, f, good, [("y", None, "is NULL"), ("y", ODDEST, "aligned"), ("ldy", 0, "stride"),
                          ("o", E, "its own"), ("w", None, "without weights")])


def test_binding_refuses_host_tensors(L):
    import torch
    t = torch.zeros((4, 16), dtype=torch.uint8)
    with pytest.raises(L.MoeError, match="host memory"):
        L.moe_quantize_mxfp4(t, L.MOE_F32, 1, 1, 1, t, 16, t, 16, stream=0)
    with pytest.raises(L.MoeError, match="host memory"):
        L.moe_collect(L.MOE_F32, 1, 1, 4, t, 4, t, None, t, 4, stream=0)
