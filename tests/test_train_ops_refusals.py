"""What the balance loss, the dense router backward, the 8-bit checkpoints and the block-scaled
FP8 product refuse, without a GPU: every call below returns its documented status before it
touches the device.  A call whose arguments are all valid reaches the device check, so on a
machine without an MI355X it returns MOE_ERR_UNSUPPORTED or MOE_ERR_HIP, never a refusal."""
import ctypes
import os

import pytest

A, B, C = (ctypes.c_void_p(4096 * i) for i in (1, 2, 3))
ODD = ctypes.c_void_p(4100)
GOOD = dict(T=256, H=256, E=16, G=4, M=2, K=4, J=2, I=128, S=1, act_dtype=1, expert_dtype=1)


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


def test_balance_loss(L):
    f = L.lib().moe_balance_loss
    need = L.lib().moe_balance_loss_workspace_bytes(P(L), 3)
    # 16 chunks of 16 tokens + 3 sequences, 16 experts, two arrays of 4 bytes
    assert need == (16 + 3) * 16 * 8
    for n in (0, -1, 1 << 22):
        bad(L, f(P(L), A, A, A, n, A, A, A, A, need, None), "n_seq")
        assert L.lib().moe_balance_loss_workspace_bytes(P(L), n) == 0
    bad(L, f(P(L, K=0), A, A, A, 3, A, A, A, A, need, None), "K=")
    for i in (0, 1, 3, 4):  # logits, topk_idx, seq_counts, seq_prob
        args = [A, A, A, A, A, A]
        for wrong, frag in ((None, "NULL"), (ODD, "aligned")):
            args[{0: 0, 1: 1, 3: 3, 4: 4}[i]] = wrong
            bad(L, f(P(L), args[0], args[1], args[2], 3, args[3], args[4], args[5], A, need,
                     None), frag)
    bad(L, f(P(L), A, A, None, 3, A, A, A, A, need, None), "seq_offsets")
    bad(L, f(P(L), A, A, A, 3, A, A, None, A, need, None), "seq_loss")
    for ws, n in ((A, need - 1), (None, need), (ODD, need)):
        bad(L, f(P(L), A, A, A, 3, A, A, A, ws, n, None), "workspace", L.MOE_ERR_WORKSPACE)


def test_balance_loss_backward(L):
    f = L.lib().moe_balance_loss_backward
    bad(L, f(P(L), A, A, 0, A, A, A, A, A, B, None), "n_seq")
    bad(L, f(P(L), None, A, 1, A, A, A, A, A, B, None), "logits is NULL")
    bad(L, f(P(L), A, None, 1, A, A, A, A, A, B, None), "seq_offsets")
    bad(L, f(P(L), A, A, 1, None, A, A, A, A, B, None), "seq_counts")
    bad(L, f(P(L), A, A, 1, A, None, A, A, A, B, None), "dseq_loss")
    bad(L, f(P(L), A, A, 1, A, A, None, A, A, B, None), "topk_idx")
    bad(L, f(P(L), A, A, 1, A, A, A, None, A, B, None), "topk_gate")
    bad(L, f(P(L), A, A, 1, A, A, A, A, A, ODD, None), "aligned")
    bad(L, f(P(L), A, A, 1, A, A, A, A, A, A, None), "over logits")


def test_router_backward_dense(L):
    f = L.lib().moe_router_backward_dense
    for kw in (dict(), dict(act_dtype=0, expert_dtype=0), dict(expert_dtype=2)):
        need = L.moe_workspace_bytes(L.problem(**{**GOOD, **kw}),
                                     L.MOE_CALL_ROUTER_BACKWARD_DENSE)
        assert need > 0
        for i in range(5):
            args = [A] * 5
            args[i] = None
            bad(L, f(P(L, **kw), *args, A, need, None), "NULL")
            args[i] = ODD
            bad(L, f(P(L, **kw), *args, A, need, None), "aligned")
        for ws, n in ((A, need - 1), (None, need), (ODD, need)):
            bad(L, f(P(L, **kw), A, A, A, A, A, ws, n, None), "workspace", L.MOE_ERR_WORKSPACE)
    bad(L, f(P(L, H=100), A, A, A, A, A, A, 1 << 30, None), "H=")
    # more threads than a launch holds
    for kw in (dict(T=(1 << 25) + 1, H=128), dict(T=(1 << 20) + 1, H=65536)):
        bad(L, f(P(L, K=1, **kw), A, A, A, A, A, A, 1 << 62, None), "2^25")


def test_checkpoints(L):
    lib = L.lib()
    fp8 = dict(expert_dtype=2)
    save, restore = lib.moe_checkpoint_save, lib.moe_checkpoint_restore
    bad(L, save(P(L, **fp8), A, B, A, None), "bf16", L.MOE_ERR_UNSUPPORTED)
    bad(L, restore(P(L, **fp8), A, A, B, C, None), "bf16", L.MOE_ERR_UNSUPPORTED)
    bad(L, save(P(L), None, B, A, None), "au is NULL")
    bad(L, save(P(L), A, ODD, A, None), "aligned")
    bad(L, save(P(L), A, B, None, None), "au_scale")
    bad(L, save(P(L), A, A, A, None), "over au")
    bad(L, restore(P(L), None, A, B, C, None), "au_q is NULL")
    bad(L, restore(P(L), A, None, B, C, None), "au_scale")
    bad(L, restore(P(L), A, A, None, None, None), "both NULL")
    bad(L, restore(P(L), A, A, ODD, None, None), "aligned")
    bad(L, restore(P(L), A, A, B, B, None), "of their own")
    bad(L, restore(P(L), A, A, A, None, None), "of their own")
    f = lib.moe_expert_ffn_backward_input_checkpoint
    for kw in (fp8, dict(act_dtype=0, expert_dtype=0)):
        bad(L, f(P(L, **kw), A, A, A, A, A, A, A, A, A, None), "BF16", L.MOE_ERR_UNSUPPORTED)
    for i in range(9):
        args = [A] * 9
        args[i] = None
        bad(L, f(P(L), *args, None), "required" if i in (0, 4) else "NULL")
    big = dict(T=30000, H=7168, E=256, G=8, M=4, K=8, J=2, I=2048)
    bad(L, f(P(L, **big), A, A, A, A, A, A, A, A, A, None), "2^31")


def test_quantize(L):
    f = L.lib().moe_quantize_fp8
    bad(L, f(A, 2, 8, 8, 8, B, 16, A, None, 0, None, None), "dtype")
    for r, c in ((0, 8), (8, 0), (-1, 8)):
        bad(L, f(A, 1, r, c, 8, B, 16, A, None, 0, None, None), "rows and cols")
    bad(L, f(A, 1, 1 << 36, 1 << 36, 1 << 36, B, 1 << 36, A, None, 0, None, None), "blocks")
    bad(L, f(A, 1, 1 << 31, 1, 1, None, 0, None, B, 1 << 31, A, None), "blocks")
    bad(L, f(A, 1, 8, 8, 7, B, 16, A, None, 0, None, None), "ldx")
    bad(L, f(None, 1, 8, 8, 8, B, 16, A, None, 0, None, None), "x is NULL")
    bad(L, f(ctypes.c_void_p(4098), 0, 8, 8, 8, B, 16, A, None, 0, None, None), "aligned")
    bad(L, f(A, 1, 8, 8, 8, None, 16, A, None, 16, A, None), "both NULL")
    for q, ld, s in ((ODD, 16, A), (B, 0, A), (B, 24, A), (B, 16, None)):
        bad(L, f(A, 1, 8, 8, 8, q, ld, s, None, 0, None, None), "q needs")
        bad(L, f(A, 1, 8, 8, 8, None, 0, None, q, ld, s, None), "qt needs")
    bad(L, f(A, 1, 8, 8, 8, A, 16, A, None, 0, None, None), "of their own")
    bad(L, f(A, 1, 8, 8, 8, B, 16, A, B, 16, A, None), "of their own")


def test_gemm(L):
    f = L.lib().moe_gemm_fp8

    def call(M=8, N=8, K=8, a=A, lda=16, sa=A, b=B, ldb=16, sb=A, rows=128, c=C, ldc=8, dt=1,
             acc=0, ws=None, n=0):
        if ws is None and n == 0:
            n = L.lib().moe_gemm_fp8_workspace_bytes(M, N, K)
            ws = A if n else None
        return f(M, N, K, a, lda, sa, b, ldb, sb, rows, c, ldc, dt, acc, ws, n, None)
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(M=(1 << 26) + 1),
               dict(N=(1 << 26) + 1), dict(N=1 << 31),
               dict(K=(1 << 22) + 1)):
        bad(L, call(**kw), "must be in")
    bad(L, call(M=1 << 26, N=(1 << 11) + 1, ldc=1 << 31), "M*N")
    for kw in (dict(a=None), dict(b=None), dict(c=None)):
        bad(L, call(**kw), "NULL")
    for kw in (dict(a=ODD), dict(b=ODD), dict(c=ODD)):
        bad(L, call(**kw), "aligned")
    for kw in (dict(sa=None), dict(sb=None)):
        bad(L, call(**kw), "a_scale and b_scale")
    for kw in (dict(lda=8), dict(ldb=24), dict(K=17, lda=16), dict(lda=(1 << 22) + 16)):
        bad(L, call(**kw), "lda and ldb")
    bad(L, call(ldc=7), "ldc")
    bad(L, call(rows=64), "b_rows")
    bad(L, call(dt=2), "c_dtype")
    bad(L, call(acc=1), "accumulate")
    bad(L, call(acc=2, dt=0), "accumulate")
    bad(L, call(c=A), "over a or b")
    bad(L, call(c=B), "over a or b")


def test_valid_calls_reach_the_device_check(L, no_gpu):
    lib = L.lib()
    n = lib.moe_gemm_fp8_workspace_bytes(8, 8, 8)
    need = lib.moe_balance_loss_workspace_bytes(P(L), 3)
    rd = L.moe_workspace_bytes(L.problem(**GOOD), L.MOE_CALL_ROUTER_BACKWARD_DENSE)
    for rc in (lib.moe_gemm_fp8(8, 8, 8, A, 16, A, B, 16, A, 1, C, 8, 0, 1, A, n, None),
               lib.moe_quantize_fp8(A, 1, 8, 8, 9, B, 16, A, C, 16, A, None),
               lib.moe_balance_loss(P(L), A, A, A, 3, A, A, A, A, need, None),
               lib.moe_balance_loss_backward(P(L), A, A, 3, A, A, None, None, None, B, None),
               lib.moe_router_backward_dense(P(L), A, A, A, A, A, A, rd, None),
               lib.moe_checkpoint_save(P(L), A, B, A, None),
               lib.moe_checkpoint_restore(P(L), A, A, None, C, None),
               lib.moe_expert_ffn_backward_input_checkpoint(P(L), A, A, A, A, A, A, A, A, A,
                                                            None)):
        assert rc in (L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_HIP), L.last_error()


def test_binding_refuses_host_and_strided_tensors(L):
    """A tensor in host memory would fault the kernel; a strided one would be read as if it
    were dense."""
    import torch
    t = torch.zeros(16)
    for call in (lambda: L.moe_checkpoint_save(L.problem(**GOOD), t, t, t),
                 lambda: L.moe_quantize_fp8(t, L.MOE_F32, 1, 16, 16, t, 16, t),
                 lambda: L.moe_gemm_fp8(1, 1, 1, t, 16, t, t, 16, t, 1, t, 1),
                 lambda: L.moe_balance_loss(L.problem(**GOOD), t, t, t, 1, t, t, t, t, 64)):
        with pytest.raises(L.MoeError, match="host memory"):
            call()
