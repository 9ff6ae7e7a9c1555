"""8-bit activation checkpoints: the codes and scales bit for bit against the definition, the
restored values exactly (a product of two fp32 numbers, rounded to the activation dtype), h
within its roundings, the expert backward from the codes bit for bit against the restored form,
and a training layer that keeps them, with the balance loss joined in, against 64 bits."""
import pytest

import workloads
from gpu_cases import TOL, case, log, make_cpu_inputs, shape_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def problem(T, K, S, I, act, H=128, E=16):
    from mixture_experts_layer_added_amd import _lib as L
    dt = L.MOE_F32 if act == "f32" else L.MOE_BF16
    return L.problem(T, H, E, 1, 1, K, 1, I, S, dt, dt)


def codes_of(x):
    """The definition: fp32 quotients, torch's cast."""
    w = x.float().view(x.shape[0], -1, 128)
    amax = w.abs().amax(2)
    scale = amax / 448
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (w / scale[:, :, None]).clamp(-448, 448).to(F8).view(torch.uint8)
    return q.view(x.shape[0], -1), scale


def values_of(q, scale, dtype):
    w = q.view(F8).float().view(q.shape[0], -1, 128) * scale[:, :, None]
    return w.view(q.shape[0], -1).to(dtype)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,S,I", [(1, 1, 0, 128), (1, 8, 1, 256), (37, 3, 1, 384),
                                     (300, 4, 0, 128), (513, 2, 1, 640)])
def test_save_and_restore(T, K, S, I, act):
    from mixture_experts_layer_added_amd import _lib as L
    dt = torch.float32 if act == "f32" else torch.bfloat16
    p, R = problem(T, K, S, I, act), T * (K + S)
    g = torch.Generator().manual_seed(T + I)
    au = torch.randn((R, 2 * I), generator=g) * 10.0 ** torch.randint(-4, 3, (R, 1), generator=g)
    au[0, :128] = 0                                  # an all-zero block
    au[R - 1, 128:256] = 0
    au[R - 1, 200] = 1e-3                            # one value in a block
    au[R // 2, 0] = -400.0                           # a large negative gate
    au = au.to(dt)
    q = torch.full((R + 1, 2 * I), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((R + 1, 2 * I // 128), -1.0, device="cuda")
    L.moe_checkpoint_save(p, au.cuda(), q, scale)
    torch.cuda.synchronize()
    rq, rs = codes_of(au)
    assert torch.equal(q[:R].cpu(), rq) and torch.equal(scale[:R].cpu(), rs)
    assert bool((q[R:] == 0x55).all()) and bool((scale[R:] == -1).all())
    # a kept value is off by at most 2^-4 of itself, or 2^-10 of the scale (half the smallest
    # code's step, 2^-9), and half a step of the type
    back, h = torch.empty((R, 2 * I), dtype=dt, device="cuda"), torch.empty((R, I), dtype=dt,
                                                                            device="cuda")
    L.moe_checkpoint_restore(p, q, scale, back, h)
    torch.cuda.synchronize()
    assert torch.equal(back.cpu(), values_of(rq, rs, dt))
    wide = rs.double().repeat_interleave(128, 1)
    eps = torch.finfo(dt).eps / 2
    off = (back.cpu().double() - au.double()).abs()
    assert bool((off <= (2 ** -4 + eps + 2 ** -23) * au.double().abs() + 2 ** -10 * wide).all())
    # h = a/(1 + exp(-a)) u: the exponential's argument a log2(e) is rounded (|a| 1.5 u), the
    # rest is a handful of roundings, u = 2^-24; then the type's half step
    a, u = back.cpu().double().chunk(2, 1)
    ref = a / (1 + torch.exp(-a)) * u
    tol = (8 + 2 * a.abs()) * 2.0 ** -24 + (0 if act == "f32" else eps)
    # where exp(-a) exceeds fp32 (2^128, a < -88.7) the quotient is 0 and the true one below
    # |a| 2^-128; below the smallest normal number, 2^-126, a result may be flushed
    tiny = 2.0 ** -126 + (a * u).abs() * 2.0 ** -128 * (a < -88.7)
    assert bool(((h.cpu().double() - ref).abs() <= tol * 1.01 * ref.abs() + tiny).all())
    # either output alone
    b2, h2 = torch.empty_like(back), torch.empty_like(h)
    L.moe_checkpoint_restore(p, q, scale, b2, None)
    L.moe_checkpoint_restore(p, q, scale, None, h2)
    torch.cuda.synchronize()
    assert torch.equal(b2, back) and torch.equal(h2, h)


def bits(t):
    return t.view(torch.int16).cpu()


@pytest.mark.parametrize("H,I,loads,S", [
    (256, 128, [0, 1, 31, 32, 33, 0], 0),      # empty groups, one row, a ragged sub-tile
    (384, 256, [64, 97, 129, 0, 200, 5], 1),   # more than one tile of 192 rows; shared rows
    (128, 384, [161, 192, 193, 3], 0),         # every sub-tile count up to six
    (256, 640, [150, 96, 10], 1),              # a last tile with idle waves
])
def test_backward_from_codes_is_the_restored_one(H, I, loads, S):
    from mixture_experts_layer_added_amd import _lib as L
    E, routed = len(loads), sum(loads)
    T = routed  # K = 1: as many tokens as routed rows
    p = problem(T, 1, S, I, "bf16", H=H, E=E)
    R, NG = T * (1 + S), E + S
    g = torch.Generator(device="cuda").manual_seed(H + I)

    def rnd(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()
    w13, w2, dy = rnd((NG, 2 * I, H), 0.05), rnd((NG, H, I), 0.05), rnd((R, H), 1.0)
    au = rnd((R, 2 * I), 1.0)
    off = torch.tensor([0] + loads).cumsum(0).tolist() + ([R] if S else [])
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    w13t, w2t = torch.empty_like(w13), torch.empty_like(w2)
    L.moe_pack_expert_weights_transposed(p, w13, w2, w13t, w2t)
    q = torch.empty((R, 2 * I), dtype=torch.uint8, device="cuda")
    scale = torch.empty((R, 2 * I // 128), device="cuda")
    L.moe_checkpoint_save(p, au, q, scale)
    back, h = torch.empty_like(au), torch.empty((R, I), dtype=au.dtype, device="cuda")
    L.moe_checkpoint_restore(p, q, scale, back, h)
    dau, dx = torch.empty_like(au), torch.empty_like(dy)
    L.moe_expert_ffn_backward_input_packed(p, off, w13t, w2t, back, dy, dau, dx)
    gau, gx, gh = (torch.full((r.shape[0] + 1, r.shape[1]), 7.0, dtype=r.dtype, device="cuda")
                   for r in (dau, dx, h))
    L.moe_expert_ffn_backward_input_checkpoint(p, off, w13t, w2t, q, scale, dy, gau, gh, gx)
    torch.cuda.synchronize()
    for got, ref, what in ((gau, dau, "dau"), (gx, dx, "dx"), (gh, h, "h")):
        assert torch.equal(bits(got[:R]), bits(ref)), what
        assert bool((got[R:] == 7).all()), what + ": a write behind the rows"
    # the first product by itself, in 64 bits: dh rounds nowhere, [da|du] once
    a, u = back.double().cpu().chunk(2, 1)
    sg = torch.sigmoid(a)
    dh, mag = torch.empty((R, I), dtype=torch.float64), torch.empty((R, I), dtype=torch.float64)
    for k in range(NG):
        lo, hi = int(off[k]), int(off[k + 1])
        d, m = dy[lo:hi].double().cpu(), w2[k].double().cpu()
        dh[lo:hi], mag[lo:hi] = d @ m, d.abs() @ m.abs()
    slope = u * sg * (1 + a * (1 - sg))
    # fp32 sums of H terms (2^-23 each), the slope's roundings and 1 - sg's cancellation
    # (64 u of |u| sg (1 + |a|)), bf16's half step
    for got, ref, big, sl in ((gau[:R, :I], dh * slope, mag, slope.abs()),
                              (gau[:R, I:], dh * a * sg, mag, (a * sg).abs())):
        tol = (H * 2.0 ** -23) * big * sl + 2.0 ** -8 * 1.01 * ref.abs() + \
            64 * 2.0 ** -24 * dh.abs() * (1 + a.abs()) * sg * (u.abs() if sl is not None else 1)\
            + 64 * 2.0 ** -24 * dh.abs() * a.abs() * sg
        assert bool(((got.cpu().double() - ref).abs() <= tol).all())
    log(f"    H={H} I={I} loads {loads} S={S}: bit-identical to the restored form")


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).abs().max() / b.abs().max().clamp(min=1e-300))


@pytest.mark.parametrize("name,gather", [("ragged-bf16", True), ("noshared-bf16", False),
                                         ("k1-j1-bf16", True), ("tiny-fp32", False),
                                         ("tiny-fp32", True), ("dense-bf16", True)])
@pytest.mark.parametrize("packed", [None, False])
def test_training_layer(name, gather, packed):
    """The layer as a training program runs it: forward, balance loss, backward with both
    gradients; against autograd in 64 bits over the same routing, with the experts'
    pre-activations replaced by the kept ones in the backward.  Bounds: those of the layer's
    other gradient tests, normwise (1e-4 fp32, 2e-2 bf16: the same rounding points)."""
    from mixture_experts_layer_added_amd.layer import MoELayer
    w = case(name)
    if packed is None and w.act == "f32":
        pytest.skip("packed weights are bf16")
    inp = make_cpu_inputs(w)
    dev = {k: v.contiguous().cuda() for k, v in inp.items()}
    args = (shape_of(w), dev["w_router"], dev["bias"], dev["w13"], dev["w2"])
    kw = dict(gather=gather, train=True, packed=packed, checkpoint8=True)
    layer = MoELayer(*args, **kw)
    other = MoELayer(*args, share=layer, **kw)  # uses the same scratch in between
    x, dy = dev["x"], workloads.make_dy(w).cuda()
    off = torch.tensor([0, w.T // 3, w.T // 3, max(w.T - 2, 0)], dtype=torch.int32, device="cuda")
    dloss = torch.tensor([0.3, 1.0, -0.2], device="cuda")
    y = layer.forward(x).clone()
    loss = layer.balance_loss(off).clone()
    other.forward(x.flip(0).contiguous())
    other.balance_loss(off)
    other.backward(dy, dseq_loss=dloss)
    layer.backward(dy, dseq_loss=dloss)
    torch.cuda.synchronize()
    plain = MoELayer(*args, gather=gather, train=True, packed=packed)
    assert torch.equal(plain.forward(x), y)

    # 64 bits, routing frozen
    idx = layer.topk_idx.long().cpu()
    X, W = inp["x"].double(), inp["w_router"].double()
    W13, W2 = inp["w13"].double(), inp["w2"].double()
    DY, T, K, E, I = dy.double().cpu(), w.T, w.K, w.E, w.I
    W.requires_grad_()
    xr = X.clone().requires_grad_()  # x as the router sees it
    z = xr @ W.t()
    s = torch.sigmoid(z.clamp(-80, 80))
    sk = s.gather(1, idx)
    gate = sk / sk.sum(1, keepdim=True)
    kept = values_of(layer.au_q.cpu(), layer.au_scale.cpu(), x.dtype).double()
    inv, Y = layer.inv_perm.long().cpu(), layer.y_sorted.double().cpu()
    dgate = (DY[:, None, :] * Y[inv]).sum(2)
    total = (gate * dgate).sum()
    o = off.tolist()
    for q in range(3):
        lo, hi = o[q], o[q + 1]
        if lo == hi:
            continue
        share = (s[lo:hi] / s[lo:hi].sum(1, keepdim=True)).mean(0)
        n = torch.bincount(idx[lo:hi].flatten(), minlength=E).double()
        lq = (n * E / (K * (hi - lo)) * share).sum()
        assert abs(float(loss[q]) - float(lq.detach())) <= 1e-5 * float(lq.detach())
        total = total + float(dloss[q]) * lq
    total.backward()
    dx, dw13, dw2 = xr.grad.clone(), torch.zeros_like(W13), torch.zeros_like(W2)
    offs = layer.offsets.tolist()
    tok = layer.sorted_token.long().cpu()
    gates = torch.ones((w.R,), dtype=torch.float64)
    gates[inv.flatten()] = gate.detach().flatten()
    for g in range(E + w.S):
        r = slice(offs[g], offs[g + 1])
        t = tok[r]
        d = gates[r, None] * DY[t]
        a, u = kept[r].chunk(2, 1)
        sg = torch.sigmoid(a)
        dh = d @ W2[g]
        da = torch.cat([dh * u * sg * (1 + a * (1 - sg)), dh * a * sg], 1)
        dw2[g], dw13[g] = d.t() @ (a * sg * u), da.t() @ X[t]
        dx.index_add_(0, t, da @ W13[g])
    errs = {k: rel(getattr(layer, k), v) for k, v in
            (("dx", dx), ("dw_router", W.grad), ("dw13", dw13), ("dw2", dw2))}
    log(f"    {name} gather={gather}: " + ", ".join(f"{k} {v:.2e}" for k, v in errs.items()))
    for k, v in errs.items():
        assert v <= TOL[w.expert], (k, v)


def test_balance_loss_of_changing_sequences():
    """Batches cut into other sequences step by step, on a stream of their own, have the losses
    and gradients of a fresh layer; a forward without its balance loss has none to go back
    through."""
    from mixture_experts_layer_added_amd.layer import MoELayer
    w = case("ragged-bf16")
    inp = make_cpu_inputs(w)
    dev = {k: v.contiguous().cuda() for k, v in inp.items()}
    args = (shape_of(w), dev["w_router"], dev["bias"], dev["w13"], dev["w2"])
    layer = MoELayer(*args, train=True)
    x, dy = dev["x"], workloads.make_dy(w).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for n in (2, 7, 1, 40, 3):
        off = torch.linspace(0, w.T, n + 1).to(torch.int32).cuda()
        dl = torch.linspace(-1, 1, n).cuda()
        torch.cuda.synchronize()
        layer.forward(x, stream=side)
        loss = layer.balance_loss(off, stream=side)
        layer.backward(dy, stream=side, dseq_loss=dl)
        with torch.cuda.stream(side):
            got.append((off, dl, loss.clone(), layer.dw_router.clone(), layer.dx.clone()))
    torch.cuda.synchronize()
    for off, dl, loss, dw, dx in got:
        fresh = MoELayer(*args, train=True)
        fresh.forward(x)
        assert torch.equal(fresh.balance_loss(off), loss)
        fresh.backward(dy, dseq_loss=dl)
        torch.cuda.synchronize()
        assert torch.equal(fresh.dw_router, dw) and torch.equal(fresh.dx, dx)
    layer.forward(x)
    with pytest.raises(AssertionError, match="balance_loss"):
        layer.backward(dy, dseq_loss=dl)
