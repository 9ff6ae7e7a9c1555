"""MoE layer object: owns the device buffers of one batch size and issues the five
C-ABI calls on the current stream.  Plumbing only (allocation and argument
marshalling); every step runs in libmoe's HIP kernels.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import torch

from . import _lib as L

_DT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16, "e4m3": L.MOE_FP8_E4M3}


@dataclass
class Shape:
    T: int
    H: int
    E: int
    G: int
    M: int
    K: int
    J: int
    I: int
    S: int = 1
    act: str = "bf16"
    expert: str = "bf16"

    def problem(self) -> L.moe_problem:
        return L.problem(self.T, self.H, self.E, self.G, self.M, self.K, self.J, self.I, self.S,
                         _DT[self.act], _DT[self.expert])

    @property
    def R(self) -> int:
        return self.T * self.K + self.S * self.T


def quantize_weights_fp8(w: torch.Tensor, stream=None):
    """bf16 [batch, rows, cols] -> (E4M3 codes uint8 [batch, rows, cols],
    fp32 scales [batch, rows/128, cols/128])."""
    assert w.dtype == torch.bfloat16 and w.dim() == 3 and w.is_contiguous()
    b, r, c = w.shape
    q = torch.empty((b, r, c), dtype=torch.uint8, device=w.device)
    s = torch.empty((b, r // 128, c // 128), dtype=torch.float32, device=w.device)
    L.moe_quantize_weights_fp8(w, q, s, b, r, c, stream)
    return q, s


def quantize_fp8(x: torch.Tensor, rows=True, cols=False):
    """fp32 or bf16 [n, m] (rows may be strided) -> E4M3 codes (uint8, row length padded to 16)
    and fp32 scales per 128: (q [n, .], scale [n, ceil(m/128)]) along the rows, (qt [m, .],
    scale_t [m, ceil(n/128)]) of the transpose; None for a form not asked for.  On the current
    stream."""
    assert x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= x.shape[1]
    assert x.dtype in (torch.bfloat16, torch.float32)
    n, m = x.shape

    def out(r, c):
        return (torch.empty((r, -(-c // 16) * 16), dtype=torch.uint8, device=x.device),
                torch.empty((r, -(-c // 128)), dtype=torch.float32, device=x.device))
    q, scale = out(n, m) if rows else (None, None)
    qt, scale_t = out(m, n) if cols else (None, None)
    L._ptrs("moe_quantize_fp8", x.as_strided((1,), (1,)))  # its device; its rows may be strided
    L.moe_quantize_fp8(x.data_ptr(), L.MOE_F32 if x.dtype == torch.float32 else L.MOE_BF16, n, m,
                       x.stride(0), q, q.shape[1] if rows else 0, scale, qt,
                       qt.shape[1] if cols else 0, scale_t)
    return q, scale, qt, scale_t


class Fp8Linear:
    """y = x W^T in block-scaled FP8 with its gradients: W [N, K] bf16 (N, K multiples of 128)
    is kept as E4M3 codes with a scale per 128 x 128 block, in both orders; x and dy are
    quantised per 128 along the dimension that each product sums over.

    forward(x [M, K] bf16) -> y [M, N] bf16; backward(dy [M, N] bf16), of the last forward, ->
    dx [M, K] bf16 and adds dy^T x to self.dw [N, K] fp32 (zero_grad clears it).  Both run on the
    current stream; the caller orders the backward's behind the forward's where they differ.
    """

    def __init__(self, w: torch.Tensor, train=False):
        self.N, self.K = w.shape
        self.train = train
        q, scale = quantize_weights_fp8(w[None])
        self.w_q, self.w_scale = q[0], scale[0]
        self.dw = None
        if train:
            self.wt_q, self.wt_scale = self.w_q.t().contiguous(), self.w_scale.t().contiguous()
            self.dw = torch.zeros((self.N, self.K), dtype=torch.float32, device=w.device)
        self._x = None

    @staticmethod
    def _gemm(a, a_scale, b, b_scale, b_rows, M, N, K, out, accumulate=0):
        n = L.moe_gemm_fp8_workspace_bytes(M, N, K)
        ws = torch.empty((n,), dtype=torch.uint8, device=a.device) if n else None
        L.moe_gemm_fp8(M, N, K, a, a.shape[1], a_scale, b, b.shape[1], b_scale, b_rows, out,
                       out.shape[1], L.MOE_F32 if out.dtype == torch.float32 else L.MOE_BF16,
                       accumulate, ws, n)
        return out

    def forward(self, x):
        M = x.shape[0]
        assert x.dtype == torch.bfloat16 and x.shape == (M, self.K)
        q, scale, qt, scale_t = quantize_fp8(x, True, self.train)
        self._x = (M, qt, scale_t)
        y = torch.empty((M, self.N), dtype=torch.bfloat16, device=x.device)
        return self._gemm(q, scale, self.w_q, self.w_scale, 128, M, self.N, self.K, y)

    def backward(self, dy):
        assert self.train, "construct the layer with train=True"
        assert self._x is not None, "call forward first"
        M, xt, xt_scale = self._x
        for t in (xt, xt_scale):  # the forward's, perhaps of another stream
            t.record_stream(torch.cuda.current_stream())
        assert dy.dtype == torch.bfloat16 and dy.shape == (M, self.N)
        q, scale, qt, scale_t = quantize_fp8(dy, True, True)
        dx = torch.empty((M, self.K), dtype=torch.bfloat16, device=dy.device)
        self._gemm(q, scale, self.wt_q, self.wt_scale, 128, M, self.K, self.N, dx)
        self._gemm(qt, scale_t, xt, xt_scale, 1, self.N, self.K, M, self.dw, 1)
        return dx

    def zero_grad(self):
        self.dw.zero_()


# batches up to this mean load per routed expert use the packed-weight GEMMs by default
PACKED_MAX_MEAN_ROWS = 160


class MoELayer:
    """Buffers for one batch of T tokens.

    Weights: w_router [E,H] fp32, bias [E] fp32 (updated in place by bias_step),
    w13 [E+S,2I,H] and w2 [E+S,H,I] in the expert dtype (uint8 E4M3 codes with
    w13_scale / w2_scale for the FP8 path).

    gather=False: permute writes x_sorted and the gate/up GEMM reads it.
    gather=True:  permute writes the index maps only (FP8: plus one quantisation of x
    per token) and the gate/up GEMM reads its rows from x through sorted_token; the
    results are identical and the permuted copy of x is never written.
    train=True (bf16 / fp32): the gate/up GEMM also keeps the pre-activations (au) and
    backward(dy) computes dx, dw_router, dw13 and dw2 (weight gradients in fp32).
    packed (bf16 and FP8 experts): the expert GEMMs run over copies of w13 and w2 in the
    library's packed layout, made once here (bf16: the same results bit for bit; with
    train, the backward input part also runs over packed copies of the transposed
    matrices, the same results bit for bit).  Default: on when the
    mean load per routed expert, T*K/E, is at most PACKED_MAX_MEAN_ROWS -- the packed
    kernels take at most 192 rows of an expert per tile (a larger expert streams its
    weights once per tile), the natural-layout kernels 256.
    checkpoint8 (with train): the pre-activations are kept between forward and backward as
    8-bit checkpoints (au_q, au_scale, written by expert_ffn_up) and h is not kept; share: another such layer of the same
    shape whose au, h, dau, dy_sorted and dx_sorted buffers this one uses too (they hold nothing
    between calls; layers that share them must not run at the same time).
    """

    def __init__(self, shape: Shape, w_router, bias, w13, w2, w13_scale=None, w2_scale=None,
                 device="cuda", gather=False, train=False, packed=None, checkpoint8=False,
                 share=None):
        assert not checkpoint8 or train, "checkpoint8 is for training"
        assert share is None or (checkpoint8 and share.checkpoint8 and share.shape == shape)
        self.checkpoint8 = checkpoint8
        self._seq_offsets = None  # of the balance loss of the last forward
        self._buffers = {}
        self.shape = shape
        self.gather = gather
        self.train = train
        can_pack = shape.act == "bf16" and shape.expert in ("bf16", "e4m3")
        if packed is None:
            packed = can_pack and shape.T * shape.K <= PACKED_MAX_MEAN_ROWS * shape.E
        self.packed = bool(packed)
        assert can_pack or not self.packed, "packed weights are built for the bf16 and FP8 paths"
        self._x = None
        self._xin = None
        self.p = shape.problem()
        self.w_router, self.bias = w_router, bias
        self.w13, self.w2, self.w13_scale, self.w2_scale = w13, w2, w13_scale, w2_scale
        self.w13p = self.w2p = self.w13tp = self.w2tp = None
        if self.packed:
            self.w13p, self.w2p = torch.empty_like(w13), torch.empty_like(w2)
            L.moe_pack_expert_weights(self.p, w13, w2, self.w13p, self.w2p)
            if train and shape.expert == "bf16":  # the backward's transposed copies
                self.w13tp, self.w2tp = torch.empty_like(w13), torch.empty_like(w2)
                L.moe_pack_expert_weights_transposed(self.p, w13, w2, self.w13tp, self.w2tp)
        T, H, E, K, R = shape.T, shape.H, shape.E, shape.K, shape.R
        act = torch.float32 if shape.act == "f32" else torch.bfloat16
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.topk_idx = torch.empty((T, K), **i32)
        self.topk_gate = torch.empty((T, K), dtype=torch.float32, device=dev)
        self.counts = torch.empty((E,), **i32)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        self.offsets = torch.empty((E + shape.S + 1,), **i32)
        self.sorted_token = torch.empty((R,), **i32)
        self.inv_perm = torch.empty((T, K), **i32)
        rows = T if gather else R  # gather: x itself (FP8: its per-token codes)
        self.x_sorted = None
        if shape.expert == "e4m3":
            self.x_q = torch.empty((rows, H), dtype=torch.uint8, device=dev)
            self.x_scale = torch.empty((rows, H // 128), dtype=torch.float32, device=dev)
        else:
            self.x_q = None if gather else torch.empty((R, H), dtype=act, device=dev)
            self.x_scale = None
        if not gather:
            self.x_sorted = self.x_q
        if shape.expert == "e4m3":
            self.h = torch.empty((R, shape.I), dtype=torch.uint8, device=dev)
            self.h_scale = torch.empty((R, shape.I // 128), dtype=torch.float32, device=dev)
        else:
            self.h = share.h if share else torch.empty((R, shape.I), dtype=act, device=dev)
            self.h_scale = None
        self.y_sorted = torch.empty((R, H), dtype=act, device=dev)
        self.y = torch.empty((T, H), dtype=act, device=dev)
        if train:
            assert shape.expert != "e4m3", "the backward is built for the bf16 and fp32 paths"
            NG, I, f32 = E + shape.S, shape.I, torch.float32
            self.au = share.au if share else torch.empty((R, 2 * I), dtype=act, device=dev)
            if checkpoint8:
                self.au_q = torch.empty((R, 2 * I), dtype=torch.uint8, device=dev)
                self.au_scale = torch.empty((R, 2 * I // 128), dtype=f32, device=dev)
            self.dy_sorted = share.dy_sorted if share else torch.empty((R, H), dtype=act,
                                                                       device=dev)
            self.dgate = torch.empty((T, K), dtype=f32, device=dev)
            self.dz = torch.empty((T, K), dtype=f32, device=dev)
            self.dx_router = torch.empty((T, H), dtype=f32, device=dev)
            self.dw_router = torch.empty((E, H), dtype=f32, device=dev)
            self.dau = share.dau if share else torch.empty((R, 2 * I), dtype=act, device=dev)
            self.dx_sorted = share.dx_sorted if share else torch.empty((R, H), dtype=act,
                                                                       device=dev)
            self.dw13 = torch.empty((NG, 2 * I, H), dtype=f32, device=dev)
            self.dw2 = torch.empty((NG, H, I), dtype=f32, device=dev)
            self.dx = torch.empty((T, H), dtype=act, device=dev)
        self.ws = {}
        for call in (L.MOE_CALL_ROUTE, L.MOE_CALL_PERMUTE):
            n = L.moe_workspace_bytes(self.p, call)
            if n == 0 and call != L.MOE_CALL_ROUTE:
                raise L.MoeError(L.MOE_ERR_INVALID_ARG, "moe_workspace_bytes", L.last_error())
            self.ws[call] = torch.empty((max(n, 256),), dtype=torch.uint8, device=dev)

    def _ws(self, call):
        t = self.ws[call]
        return t, t.numel()

    def _grown(self, name, n, dtype, stream):
        """The first n elements of a buffer that is made on its first use, on the stream that
        uses it, and made larger when n passes it.  Outgrown ones are kept: work that reads
        them may still be in flight, on whatever stream."""
        held = self._buffers.setdefault(name, [])
        if not held or held[-1].numel() < n:
            size = max(n, 2 * held[-1].numel()) if held else n
            held.append(self._fresh(size, dtype, stream))
        return held[-1][:n]

    def _fresh(self, n, dtype, stream):
        """n elements allocated on the stream that uses them."""
        with (contextlib.nullcontext() if stream is None else
              torch.cuda.stream(torch.cuda.ExternalStream(L._stream(stream)))):
            return torch.empty((n,), dtype=dtype, device=self.logits.device)

    def route(self, x, stream=None):
        self._seq_offsets = None
        L.moe_route(self.p, x, self.w_router, self.bias, self.topk_idx, self.topk_gate,
                    self.counts, self.logits, None, 0, stream)

    def permute(self, x, stream=None):
        ws, n = self._ws(L.MOE_CALL_PERMUTE)
        if self.gather:
            L.moe_permute(self.p, x, self.topk_idx, self.offsets, self.sorted_token,
                          self.inv_perm, None, None, ws, n, stream)
            if self.shape.expert == "e4m3":
                L.moe_quantize_act_fp8(self.p, x, self.x_q, self.x_scale, stream)
            self._x = x
        else:
            L.moe_permute(self.p, x, self.topk_idx, self.offsets, self.sorted_token,
                          self.inv_perm, self.x_sorted, self.x_scale, ws, n, stream)
            self._xin = x

    def expert_ffn_up(self, stream=None):
        if self.packed:
            if self.shape.expert == "e4m3":
                xin, st = (self.x_q, self.sorted_token) if self.gather else (self.x_sorted, None)
            else:
                xin, st = (self._x, self.sorted_token) if self.gather else (self.x_sorted, None)
            L.moe_expert_ffn_up_packed(self.p, xin, self.x_scale, st, self.offsets, self.w13,
                                       self.w13p, self.w13_scale, self.h, self.h_scale,
                                       self.au if self.train else None, stream)
        elif self.train:
            xin, st = (self._x, self.sorted_token) if self.gather else (self.x_sorted, None)
            L.moe_expert_ffn_up_save(self.p, xin, st, self.offsets, self.w13, self.h, self.au,
                                     stream)
        elif self.gather:
            xin = self.x_q if self.shape.expert == "e4m3" else self._x
            L.moe_expert_ffn_up_gather(self.p, xin, self.x_scale, self.sorted_token,
                                       self.offsets, self.w13, self.w13_scale, self.h,
                                       self.h_scale, stream)
        else:
            L.moe_expert_ffn_up(self.p, self.x_sorted, self.x_scale, self.offsets, self.w13,
                                self.w13_scale, self.h, self.h_scale, stream)
        if self.checkpoint8:  # here, so that a forward of single calls keeps its own batch's too
            L.moe_checkpoint_save(self.p, self.au, self.au_q, self.au_scale, stream)

    def expert_ffn_down(self, stream=None):
        if self.packed:
            L.moe_expert_ffn_down_packed(self.p, self.h, self.h_scale, self.offsets, self.w2p,
                                         self.w2_scale, self.y_sorted, stream)
            return
        L.moe_expert_ffn_down(self.p, self.h, self.h_scale, self.offsets, self.w2, self.w2_scale,
                              self.y_sorted, stream)

    def expert_ffn(self, stream=None):
        self.expert_ffn_up(stream)
        self.expert_ffn_down(stream)

    def combine(self, stream=None):
        L.moe_combine(self.p, self.y_sorted, self.inv_perm, self.topk_gate, self.y, stream)

    def forward(self, x, stream=None):
        """route -> permute -> expert FFN -> combine; returns self.y (overwritten by the
        next call)."""
        self.route(x, stream)
        self.permute(x, stream)
        self.expert_ffn(stream)
        self.combine(stream)
        return self.y

    def bias_step(self, gamma=0.01, stream=None):
        """Aux-loss-free bias update from this batch's expert counts (in place)."""
        L.moe_bias_update(self.p, self.counts, gamma, self.bias, stream)

    def balance_loss(self, seq_offsets, stream=None):
        """Sequence-wise balance loss of the last forward's routing: seq_offsets [n_seq+1] int32
        on the device -> [n_seq] fp32, a tensor of its own.  Also kept, until the next call:
        counts per (sequence, expert) and mean affinity shares in self.seq_counts,
        self.seq_prob.  Its gradient joins the next backward(dy, dseq_loss=...)."""
        assert seq_offsets.dtype == torch.int32 and seq_offsets.dim() == 1
        n, E, f32 = seq_offsets.numel() - 1, self.shape.E, torch.float32
        need = L.moe_balance_loss_workspace_bytes(self.p, n)
        ws = self._grown("balance_ws", need, torch.uint8, stream)
        loss = self._fresh(n, f32, stream)
        self.seq_counts = self._grown("seq_counts", n * E, torch.int32, stream).view(n, E)
        self.seq_prob = self._grown("seq_prob", n * E, f32, stream).view(n, E)
        L.moe_balance_loss(self.p, self.logits, self.topk_idx, seq_offsets, n, self.seq_counts,
                           self.seq_prob, loss, ws, need, stream)
        self._seq_offsets = seq_offsets
        return loss

    def router_backward_dense(self, dseq_loss, stream=None):
        """The router's backward with the balance loss's gradient (dseq_loss [n_seq] fp32, the
        gradient of the sequences' losses) joined to the gates'."""
        assert self._seq_offsets is not None, "call balance_loss after the forward first"
        n_seq = self._seq_offsets.numel() - 1
        assert dseq_loss.dtype == torch.float32 and dseq_loss.shape == (n_seq,)
        T, E = self.shape.T, self.shape.E
        self.dlogits = self._grown("dlogits", T * E, torch.float32, stream).view(T, E)
        L.moe_balance_loss_backward(self.p, self.logits, self._seq_offsets, n_seq,
                                    self.seq_counts, dseq_loss, self.topk_idx, self.topk_gate,
                                    self.dgate, self.dlogits, stream)
        x = self._x if self.gather else self._xin
        n = L.moe_workspace_bytes(self.p, L.MOE_CALL_ROUTER_BACKWARD_DENSE)
        ws = self._grown("dense_ws", n, torch.uint8, stream)
        L.moe_router_backward_dense(self.p, x, self.w_router, self.dlogits, self.dx_router,
                                    self.dw_router, ws, n, stream)

    def expert_ffn_backward_input(self, stream=None):
        if self.checkpoint8 and self.w13tp is not None:
            L.moe_expert_ffn_backward_input_checkpoint(
                self.p, self.offsets, self.w13tp, self.w2tp, self.au_q, self.au_scale,
                self.dy_sorted, self.dau, self.h, self.dx_sorted, stream)
            return
        if self.checkpoint8:
            L.moe_checkpoint_restore(self.p, self.au_q, self.au_scale, self.au, self.h, stream)
        if self.w13tp is not None:
            L.moe_expert_ffn_backward_input_packed(self.p, self.offsets, self.w13tp, self.w2tp,
                                                   self.au, self.dy_sorted, self.dau,
                                                   self.dx_sorted, stream)
            return
        L.moe_expert_ffn_backward_input(self.p, self.offsets, self.w13, self.w2, self.au,
                                        self.dy_sorted, self.dau, self.dx_sorted, stream)

    def expert_ffn_backward_weight(self, stream=None):
        xin, st = (self._x, self.sorted_token) if self.gather else (self.x_sorted, None)
        L.moe_expert_ffn_backward_weight(self.p, xin, st, self.offsets, self.h, self.dy_sorted,
                                         self.dau, self.dw13, self.dw2, stream)

    def combine_backward(self, dy, stream=None):
        L.moe_combine_backward(self.p, dy, self.y_sorted, self.inv_perm, self.topk_gate,
                               self.dy_sorted, self.dgate, stream)

    def router_backward(self, stream=None):
        x = self._x if self.gather else self._xin
        L.moe_router_backward(self.p, x, self.w_router, self.logits, self.topk_idx,
                              self.topk_gate, self.dgate, self.offsets, self.sorted_token,
                              self.dz, self.dx_router, self.dw_router, stream)

    def unpermute_sum(self, stream=None):
        L.moe_unpermute_sum(self.p, self.dx_sorted, self.inv_perm, self.dx_router, self.dx,
                            stream)

    def backward(self, dy, stream=None, dseq_loss=None):
        """Gradients of sum(dy * y) for the last forward (train=True), plus those of
        sum(dseq_loss * balance_loss(...)) where dseq_loss is given: returns self.dx and
        fills dw_router, dw13, dw2 (fp32).  The routing bias has no gradient."""
        assert self.train, "construct the layer with train=True"
        self.combine_backward(dy, stream)
        if dseq_loss is None:
            self.router_backward(stream)
        else:
            self.router_backward_dense(dseq_loss, stream)
        self.expert_ffn_backward_input(stream)
        self.expert_ffn_backward_weight(stream)
        self.unpermute_sum(stream)
        return self.dx

    def step(self, x, gamma=0.01, stream=None):
        y = self.forward(x, stream)
        self.bias_step(gamma, stream)
        return y
