"""The layers made of the MXFP4 calls and of a share of the experts: a linear layer with its
gradients, the MoE layer with 4-bit experts, and shares whose outputs add up to the layer's.

Tolerances: products of quantised operands as in test_gpu_mxfp4 (exact products, fp32 sums); the fp32
and bf16 expert products within the bounds that the layer's tests hold them to, 1e-4 and 2e-2 of the
largest value."""
import pytest

import workloads
from gpu_cases import TOL, shape_of
from mxfp4_cases import quantize, values
from test_gpu_mxfp4 import check_experts, check_product

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def mx(x, random=None):
    """x as the values of its MXFP4 form, in 64 bits."""
    return values(*quantize(x, random), x.shape[1])


# ---------------------------------------------------------------------------
# linear layer
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,N,K", [(1, 64, 96), (37, 130, 70), (300, 256, 512)])
def test_linear(M, N, K):
    from mixture_experts_layer_added_amd.layer import Fp4Linear
    g = torch.Generator().manual_seed(N)
    x, w = torch.randn((M, K), generator=g).bfloat16(), torch.randn((N, K), generator=g).bfloat16()
    dy = torch.randn((M, N), generator=g).bfloat16()
    r = torch.randint(0, 256, (M, N), generator=g, dtype=torch.uint8)
    lin = Fp4Linear(w.cuda(), train=True)
    y = lin.forward(x.cuda())
    dx = lin.backward(dy.cuda(), r.cuda())
    dw = lin.dw.clone()
    lin.forward(x.cuda())
    lin.backward(dy.cuda(), r.cuda())  # adds to dw
    torch.cuda.synchronize()
    check_product(y.cpu(), mx(x), mx(w))
    check_product(dx.cpu(), mx(dy, r), mx(w.t()))
    check_product(dw.cpu(), mx(dy.t(), r.t()), mx(x.t()))
    check_product(lin.dw.cpu(), mx(dy.t(), r.t()), mx(x.t()), dw.cpu())
    near = Fp4Linear(w.cuda(), train=True, stochastic=False)
    near.forward(x.cuda())
    check_product(near.backward(dy.cuda()).cpu(), mx(dy), mx(w.t()))
    lin.zero_grad()
    torch.cuda.synchronize()
    assert not bool(lin.dw.any())


def test_linear_draws_its_bytes():
    """Without given bytes two backward passes round differently."""
    from mixture_experts_layer_added_amd.layer import Fp4Linear
    g = torch.Generator().manual_seed(0)
    lin = Fp4Linear(torch.randn((128, 128), generator=g).bfloat16().cuda(), train=True)
    x, dy = (torch.randn((64, 128), generator=g).bfloat16().cuda() for _ in range(2))
    lin.forward(x)
    a, b = lin.backward(dy).clone(), lin.backward(dy)
    torch.cuda.synchronize()
    assert not torch.equal(a, b)


def test_linear_step_captured():
    """A training step in a graph, replayed on new inputs, against the eager step."""
    from mixture_experts_layer_added_amd.layer import Fp4Linear
    g = torch.Generator().manual_seed(3)
    M, N, K = 200, 256, 320
    w = torch.randn((N, K), generator=g).bfloat16().cuda()
    lin, eager = Fp4Linear(w, train=True), Fp4Linear(w, train=True)
    x, dy = torch.zeros((M, K), device="cuda").bfloat16(), torch.zeros((M, N), device="cuda").bfloat16()
    r = torch.zeros((M, N), dtype=torch.uint8, device="cuda")

    def step(layer):
        layer.zero_grad()
        y = layer.forward(x)
        return y, layer.backward(dy, r)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(lin)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = step(lin)
    for _ in range(3):
        x.copy_(torch.randn((M, K), generator=g))
        dy.copy_(torch.randn((M, N), generator=g))
        r.copy_(torch.randint(0, 256, (M, N), generator=g, dtype=torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), dx.clone(), lin.dw.clone()
        want = *step(eager), eager.dw
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_helpers():
    from mixture_experts_layer_added_amd.layer import dequantize_mxfp4, quantize_mxfp4
    x = torch.randn((40, 300), generator=torch.Generator().manual_seed(1))
    part = x.cuda()[:, 7:207]  # strided rows that begin anywhere
    q, s, qt, st = quantize_mxfp4(part, True, True)
    a, b = dequantize_mxfp4(q, s, 200, torch.float32), dequantize_mxfp4(qt, st, 40)
    torch.cuda.synchronize()
    assert torch.equal(a.cpu().double(), mx(x[:, 7:207]))
    assert torch.equal(b.cpu().double(), mx(x[:, 7:207].t()))


# ---------------------------------------------------------------------------
# the MoE layer with 4-bit experts
# ---------------------------------------------------------------------------
def make_layer(T=300, S=1, **kw):
    from mixture_experts_layer_added_amd.layer import MoELayer, quantize_weights_mxfp4
    w = workloads.get("v3-bf16", **{**dict(T=T, H=384, E=16, G=4, M=2, K=4, J=2, I=256, S=S), **kw})
    W = {k: v.cuda() for k, v in workloads.make_weights(w).items()}
    shape = shape_of(w)
    shape.expert = "mxfp4"
    q13, q2 = quantize_weights_mxfp4(W["w13"] * 16), quantize_weights_mxfp4(W["w2"] * 16)
    layer = MoELayer(shape, W["w_router"], W["bias"].clone(), q13[0], q2[0], q13[1], q2[1])
    return w, W, q13, q2, layer, workloads.make_x(w).cuda()


@pytest.mark.parametrize("T,S", [(300, 1), (1, 1), (37, 0)])
def test_layer(T, S):
    w, W, q13, q2, layer, x = make_layer(T, S)
    y = layer.step(x)
    torch.cuda.synchronize()
    off = layer.offsets.cpu().tolist()
    X = mx(x.cpu().float())
    assert torch.equal(values(layer.x_q, layer.x_scale, w.H), X)
    r = dict(off=off, token=layer.sorted_token.cpu().long(), X=X, hq=layer.h.cpu(),
             hs=layer.h_scale.cpu(), y=layer.y_sorted.cpu(),
             W13=[values(a, b, w.H) for a, b in zip(q13[0], q13[1])],
             W2=[values(a, b, w.I) for a, b in zip(q2[0], q2[1])])
    r["hs"][:, w.I // 32:] = 0x55  # what the check expects of bytes that nothing writes
    check_experts(r, w.H, w.I)
    ys, row = layer.y_sorted.cpu().double(), layer.inv_perm.cpu().long()
    gate = layer.topk_gate.cpu().double()
    want = (ys[row] * gate[:, :, None]).sum(1)
    size = (ys[row] * gate[:, :, None]).abs().sum(1)
    if S:
        want, size = want + ys[T * w.K:], size + ys[T * w.K:].abs()
    err = (y.cpu().double() - want).abs()
    assert bool((err <= (w.K + 2) * 2.0 ** -24 * size + 2.0 ** -8 * want.abs() * 1.001).all())


def test_layer_refuses():
    from mixture_experts_layer_added_amd.layer import MoELayer
    w, W, q13, q2, layer, x = make_layer(20)
    with pytest.raises(AssertionError):
        MoELayer(layer.shape, W["w_router"], W["bias"], q13[0], q2[0], q13[1], q2[1], train=True)


# ---------------------------------------------------------------------------
# shares of the experts
# ---------------------------------------------------------------------------
def test_shares_add_up_to_the_layer():
    """The 4-bit layer without a shared expert against the sum of three shares of its experts: the
    rows are the same bit for bit, each share's sum is rounded once more."""
    from mixture_experts_layer_added_amd.layer import ExpertShare
    w, W, q13, q2, layer, x = make_layer(260, 0)
    y = layer.forward(x).double()
    idx, gate = layer.topk_idx, layer.topk_gate
    total, size = 0, 0
    for lo, hi in ((0, 3), (3, 12), (12, 16)):
        share = ExpertShare(lo, q13[0][lo:hi].contiguous(), q2[0][lo:hi].contiguous(),
                            q13[1][lo:hi].contiguous(), q2[1][lo:hi].contiguous(), "mxfp4")
        part = share.forward(x, idx, gate).double()
        total, size = total + part, size + part.abs()
    torch.cuda.synchronize()
    assert bool(((total - y).abs() <= 2.0 ** -8 * (size + y.abs()) * 1.01 + 1e-30).all())


def reference(x, idx, gate, first, w13, w2, dy):
    """y, dx, dgate, dw13, dw2 of a share from the formulas, in 64 bits."""
    T, K = idx.shape
    I = w2.shape[2]
    x, gate, w13, w2, dy = (t.double() for t in (x, gate, w13, w2, dy))
    y, dx, dg = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(gate)
    d13, d2 = torch.zeros_like(w13), torch.zeros_like(w2)
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k]) - first
            if not 0 <= e < len(w13):
                continue
            au = w13[e] @ x[t]
            a, u = au[:I], au[I:]
            s = torch.sigmoid(a)
            h = a * s * u
            out = w2[e] @ h
            y[t] += gate[t, k] * out
            dg[t, k] = dy[t] @ out
            do = gate[t, k] * dy[t]
            dh = w2[e].t() @ do
            d2[e] += torch.outer(do, h)
            dau = torch.cat([dh * u * (s + a * s * (1 - s)), dh * a * s])
            d13[e] += torch.outer(dau, x[t])
            dx[t] += w13[e].t() @ dau
    return y, dx, dg, d13, d2


def share_inputs(T, K, E, H, I, count, seed, act):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = torch.float32 if act == "f32" else torch.bfloat16
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    return (n(T, H).to(dt), idx, torch.softmax(n(T, K), 1), (n(count, 2 * I, H) * 0.05).to(dt),
            (n(count, H, I) * 0.05).to(dt), n(T, H).to(dt))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,E,first,count", [(1, 2, 4, 1, 2), (40, 4, 12, 3, 5), (33, 3, 6, 0, 6),
                                               (20, 2, 64, 60, 4), (9, 2, 4, 4, 3)])
def test_share_with_gradients(T, K, E, first, count, act):
    from mixture_experts_layer_added_amd.layer import ExpertShare
    H, I = 128, 128
    x, idx, gate, w13, w2, dy = share_inputs(T, K, E, H, I, count, T + E, act)
    share = ExpertShare(first, w13.cuda(), w2.cuda(), expert=act, train=True)
    y = share.forward(x.cuda(), idx.cuda(), gate.cuda())
    dx, dg = share.backward(dy.cuda())
    torch.cuda.synchronize()
    want = reference(x, idx, gate, first, w13, w2, dy)
    for got, ref in zip((y, dx, dg, share.dw13, share.dw2), want):
        err = (got.cpu().double() - ref).abs().max()
        assert err <= TOL[act] * ref.abs().max(), (err, ref.abs().max())
    quiet = ExpertShare(first, w13.cuda(), w2.cuda(), expert=act)
    assert torch.equal(quiet.forward(x.cuda(), idx.cuda(), gate.cuda()), y)


def test_share_gradients_by_differences():
    """The fp32 share's gradients against central differences of its forward along random ways."""
    from mixture_experts_layer_added_amd.layer import ExpertShare
    x, idx, gate, w13, w2, dy = share_inputs(12, 3, 6, 128, 128, 3, 5, "f32")
    x, idx, gate, w13, w2, dy = (t.cuda() for t in (x, idx, gate, w13, w2, dy))
    share = ExpertShare(2, w13, w2, expert="f32", train=True)
    share.forward(x, idx, gate)
    dx, dg = share.backward(dy)
    grads = dict(x=dx, gate=dg, w13=share.dw13.clone(), w2=share.dw2.clone())
    base = dict(x=x, gate=gate, w13=w13, w2=w2)
    g = torch.Generator().manual_seed(1)
    for name, v in base.items():
        way = torch.randn(v.shape, generator=g).cuda()
        way = way * (v.abs().mean() / way.abs().mean())
        f = []
        for sign in (1, -1):
            a = {**base, name: v + sign * 2.0 ** -6 * way}
            s = ExpertShare(2, a["w13"], a["w2"], expert="f32")
            f.append((s.forward(a["x"], idx, a["gate"]).double() * dy.double()).sum())
        slope, want = (f[0] - f[1]) * 2.0 ** 5, (grads[name].double() * way.double()).sum()
        # third order of the step (2^-12 of the slope's scale) and fp32's error of f over the step
        scale = (grads[name].double().abs() * way.double().abs()).sum()
        assert abs(slope - want) <= 2.0 ** -8 * scale, name


@pytest.mark.parametrize("expert", ["bf16", "mxfp4"])
def test_share_without_tokens(expert):
    from mixture_experts_layer_added_amd.layer import ExpertShare, quantize_weights_mxfp4
    x, idx, gate, w13, w2, dy = share_inputs(5, 2, 4, 128, 128, 2, 1, "bf16")
    w13, w2 = w13.cuda(), w2.cuda()
    if expert == "mxfp4":
        (a, sa), (b, sb) = quantize_weights_mxfp4(w13), quantize_weights_mxfp4(w2)
        share = ExpertShare(0, a, b, sa, sb, "mxfp4")
    else:
        share = ExpertShare(0, w13, w2, train=True)
    none = share.forward(x[:0].cuda(), idx[:0].cuda(), gate[:0].cuda())
    assert none.shape == (0, 128)
    if expert == "bf16":
        dx, dg = share.backward(dy[:0].cuda())
        assert dx.shape == (0, 128) and dg.shape == (0, 2) and not bool(share.dw13.any())
    away = torch.full_like(idx, 9).cuda()  # tokens, none of whose choices is here
    y = share.forward(x.cuda(), away, gate.cuda())
    torch.cuda.synchronize()
    assert not bool(y.any())
    if expert == "bf16":
        dx, dg = share.backward(dy.cuda())
        torch.cuda.synchronize()
        assert not bool(dx.any() or dg.any() or share.dw13.any() or share.dw2.any())


def test_share_captured():
    """A 4-bit share's forward in a graph, replayed on new tokens and choices."""
    from mixture_experts_layer_added_amd.layer import ExpertShare, quantize_weights_mxfp4
    T, K, E, count = 90, 4, 24, 8
    x, idx, gate, w13, w2, _ = share_inputs(T, K, E, 256, 128, count, 2, "bf16")
    (a, sa), (b, sb) = quantize_weights_mxfp4(w13.cuda()), quantize_weights_mxfp4(w2.cuda())
    share = ExpertShare(8, a, b, sa, sb, "mxfp4")
    x, idx, gate = x.cuda(), idx.cuda(), gate.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        share.forward(x, idx, gate)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = share.forward(x, idx, gate)
    g = torch.Generator().manual_seed(7)
    for _ in range(4):
        x.copy_(torch.randn(x.shape, generator=g))
        idx.copy_(torch.randint(0, E, idx.shape, generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        want = share.forward(x, idx, gate)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
