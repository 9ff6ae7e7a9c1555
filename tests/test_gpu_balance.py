"""The sequence-wise balance loss, its counts and its gradient, and the router's backward for a
dense logit gradient, against their definitions in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32 relative to the value):
- an affinity s and its complement 1 - s: an exponential of a few u, an add, a reciprocal and a
  product, 8 u relative (all terms are positive); a token's sum over E <= 512 experts adds at
  most 8 in a lane and 6 across lanes, 14 more; a share s/S 8 + 22 + 2 = 32 u.
- P: 32 u and one u per addition in the longest chain: at most 64 in a lane, 6 + 2 across the
  workgroup, then a sequence's slots, one per 8 tokens or more: (128 + L/8) u relative.
- the loss: a sum of E positive products f P, 4 u each: 32 u more.
- the gradient (c - m)/S s(1-s): the bracket may cancel, so the error is counted against
  (|c| + m)/S s(1-s): c 8 u, m 32 + 14 + 8, 1/S 24, the slope 16, and the products: 128 u.  The
  gates' part is counted against (|dg| + sum |g dg|)/sum s_k s(1-s): 16 terms, 128 u.
- the dense products: fp32 operands of which at most 2^-24 is dropped on either side, a product
  and one rounding or truncation (2^-23) per addition: (n + 16) 2^-23 sum |a b|.
"""
import numpy as np
import pytest

from gpu_cases import log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def problem(T, E, K, H=128, act="bf16"):
    from mixture_experts_layer_added_amd import _lib as L
    dt = L.MOE_F32 if act == "f32" else L.MOE_BF16
    return L.problem(T, H, E, 1, 1, K, 1, 128, 0, dt, dt)


def inputs(T, E, K, seed, spread=1.7):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((T, E), generator=g) * spread
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int()
    dgate = torch.randn((T, K), generator=g) * 0.01
    return z, idx, dgate


def reference(z, idx, off, dloss, dgate=None):
    """counts, P, loss, gradient and the scale that the gradient's error is counted against."""
    z, T, E = z.double(), *z.shape
    K, n = idx.shape[1], len(off) - 1
    s = 1 / (1 + torch.exp(-z.clamp(-80, 80)))
    slope = torch.where(z.abs() > 80, 0.0, s / (1 + torch.exp(z.clamp(-80, 80))))
    counts = torch.zeros((n, E), dtype=torch.int32)
    prob, loss = torch.zeros((n, E), dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    grad, mag = torch.zeros_like(z), torch.zeros_like(z)
    for q in range(n):
        lo, hi = off[q], off[q + 1]
        if lo == hi:
            continue
        share = s[lo:hi] / s[lo:hi].sum(1, keepdim=True)
        counts[q] = torch.bincount(idx[lo:hi].flatten().long(), minlength=E).int()
        f = counts[q].double() * E / (K * (hi - lo))
        prob[q] = share.sum(0) / (hi - lo)
        loss[q] = (f * prob[q]).sum()
        c = (f * float(dloss[q]) / (hi - lo))[None]
        m, top = (c * share).sum(1, keepdim=True), s[lo:hi].sum(1, keepdim=True)
        grad[lo:hi] = (c - m) / top * slope[lo:hi]
        mag[lo:hi] = (c.abs() + (c * share).abs().sum(1, keepdim=True)) / top * slope[lo:hi]
    if dgate is not None:
        at = idx.long()
        sk, dg = s.gather(1, at), dgate.double()
        gate = (sk / sk.sum(1, keepdim=True)).float().double()  # as the router stores it
        dk = (dg - (gate * dg).sum(1, keepdim=True)) / sk.sum(1, keepdim=True)
        mk = (dg.abs() + (gate * dg).abs().sum(1, keepdim=True)) / sk.sum(1, keepdim=True)
        grad.scatter_add_(1, at, dk * slope.gather(1, at))
        mag.scatter_add_(1, at, mk * slope.gather(1, at))
    return counts, prob, loss, grad, mag


def gates(z, idx):
    s = torch.sigmoid(z.double().clamp(-80, 80)).gather(1, idx.long())
    return (s / s.sum(1, keepdim=True)).float()


class Balance:
    """The two calls on buffers that are filled with rubbish first."""

    def __init__(self, z, idx, off, dloss, dgate=None):
        from mixture_experts_layer_added_amd import _lib as L
        self.L, (T, E), K, n = L, z.shape, idx.shape[1], len(off) - 1
        self.p, self.n = problem(T, E, K), n
        self.z, self.idx = z.cuda(), idx.cuda()
        self.off = torch.tensor(off, dtype=torch.int32).cuda()
        self.dloss = dloss.cuda()
        self.dgate = None if dgate is None else dgate.cuda()
        self.gate = gates(z, idx).cuda()
        self.counts = torch.full((n, E), -7, dtype=torch.int32, device="cuda")
        self.prob = torch.full((n, E), float("nan"), device="cuda")
        self.loss = torch.full((n,), float("nan"), device="cuda")
        self.dz = torch.full((T, E), float("nan"), device="cuda")
        size = L.moe_balance_loss_workspace_bytes(self.p, n)
        self.ws = torch.full((size + 256,), 0x7f, dtype=torch.uint8, device="cuda")
        self.size = size

    def __call__(self, stream=None):
        L = self.L
        L.moe_balance_loss(self.p, self.z, self.idx, self.off, self.n, self.counts, self.prob,
                           self.loss, self.ws, self.size, stream)
        L.moe_balance_loss_backward(self.p, self.z, self.off, self.n, self.counts, self.dloss,
                                    self.idx, self.gate, self.dgate, self.dz, stream)

    def outputs(self):
        torch.cuda.synchronize()
        assert bool((self.ws[self.size:] == 0x7f).all()), "a write behind the workspace"
        return [t.cpu() for t in (self.counts, self.prob, self.loss, self.dz)]


def check(z, idx, off, dgate=None, tag="", seed=5):
    n = len(off) - 1
    dloss = torch.randn((n,), generator=torch.Generator().manual_seed(seed))
    b = Balance(z, idx, off, dloss, dgate)
    b()
    counts, prob, loss, dz = b.outputs()
    rc, rp, rl, rg, mag = reference(z, idx, off, dloss, dgate)
    assert torch.equal(counts, rc), tag
    length = torch.tensor([hi - lo for lo, hi in zip(off[:-1], off[1:])]).double()
    tol = (128 + length / 8) * U
    assert bool(((prob.double() - rp).abs() <= tol[:, None] * rp).all()), tag
    assert bool(((loss.double() - rl).abs() <= (tol + 32 * U) * rl).all()), tag
    err = (dz.double() - rg).abs()
    assert bool((err <= 128 * U * mag).all()), (tag, float((err / mag.clamp(min=1e-300)).max() / U))
    log(f"    {tag}: {n} sequences, gradient within {float((err / mag.clamp(min=1e-300)).max() / U):.1f} u")
    return counts, prob, loss, dz


@pytest.mark.parametrize("E", [1, 3, 4, 8, 16, 30, 32, 48, 64, 100, 128, 250, 256, 257, 384, 510,
                               512])
def test_expert_counts(E):
    """Every lane layout, expert counts that fill none, and K from 1 to 16."""
    K = min(E, 1 + E % 16)
    for T in (77, 600):  # one launch and two
        z, idx, dgate = inputs(T, E, K, seed=E + T)
        check(z, idx, [0, 40, 40, T - 9], dgate, f"E={E} K={K} T={T}")


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 63, 300, 512, 513, 1000, 8193, 17001])
def test_token_counts(T):
    """One token to more than a chunk per compute unit; ragged cuts, empty sequences."""
    E, K = 64, 6
    z, idx, dgate = inputs(T, E, K, seed=T)
    check(z, idx, [0, T], None, f"T={T} one sequence")
    cuts = np.sort(np.random.default_rng(T).integers(0, T + 1, size=9)).tolist()
    check(z, idx, [0, 0] + cuts + [T, T], dgate, f"T={T} ragged")


@pytest.mark.parametrize("T,E", [(65536, 32), (65536, 48), (40003, 64), (70001, 50),
                                 (65537, 300)])
def test_long_batch(T, E):
    """64-token chunks, two or eight tokens a lane group in the backward; sequences that begin
    and end inside chunks, and inside a lane group's tokens."""
    K = 4
    g = torch.Generator().manual_seed(2)
    z = torch.randn((T, E), generator=g)
    idx = torch.rand((T, E), generator=g).topk(K, dim=1).indices.int()
    dgate = torch.randn((T, K), generator=g)
    check(z, idx, [0, 1, 63, 64, 200, 39000, 39001, T - 500], dgate, f"{T} tokens E={E}")


def test_one_token_sequences():
    T, E, K = 130, 24, 3
    z, idx, dgate = inputs(T, E, K, seed=4)
    check(z, idx, list(range(T + 1)), dgate, "one token each")


def test_padding_rows():
    """Tokens before the first and behind the last sequence belong to none: they are not
    counted, and get a zero gradient, or the gates' part alone."""
    T, E, K = 100, 16, 4
    z, idx, dgate = inputs(T, E, K, seed=6)
    dz = check(z, idx, [10, 30, 30, 77], None, "padding")[3]
    assert not dz[:10].any() and not dz[77:].any() and dz[10:77].any()
    check(z, idx, [10, 30, 30, 77], dgate, "padding with gates")
    counts, prob, loss, dz = check(z, idx, [0, 0], None, "no token in any sequence")
    assert not counts.any() and not prob.any() and not loss.any() and not dz.any()


def test_saturated_logits():
    """Logits at and past the clamp, all equal, and far apart: no overflow, no gradient where
    the clamp is flat, and affinities whose complement cancels in fp32."""
    T, E, K = 24, 32, 4
    z, idx, dgate = inputs(T, E, K, seed=8)
    z[0] = 80.0
    z[1] = -80.0
    z[2] = 81.0
    z[3] = -200.0
    z[4] = 3e38
    z[5] = torch.linspace(-100, 100, E)
    z[6] = 0.0
    z[7] = 20.0
    z[8] = -60.0
    z[9, ::2] = 79.0
    dz = check(z, idx, [0, 5, 24], dgate, "saturated")[3]
    assert not dz[2:5].any()


def test_uniform_loads_give_one():
    """With every expert chosen equally often, or every share equal, the loss is 1."""
    T, E, K = 64, 8, 2
    z, _, _ = inputs(T, E, K, seed=9)
    idx = torch.stack([torch.tensor([(2 * t) % E, (2 * t + 1) % E]) for t in range(T)]).int()
    loss, dz = check(z, idx, [0, T], None, "uniform loads")[2:]
    assert abs(float(loss[0]) - 1) <= (160 + T / 8) * U
    assert not dz.any()  # every c[e] is the same: nothing to gain
    loss = check(torch.zeros_like(z), torch.zeros_like(idx), [0, T], None, "uniform shares")[2]
    assert abs(float(loss[0]) - 1) <= (160 + T / 8) * U


def test_same_index_twice_and_indices_out_of_range():
    """A caller's own indices: one expert chosen twice by a token counts twice; an index outside
    [0, E) is not counted and takes no gradient."""
    T, E, K = 40, 16, 4
    z, idx, dgate = inputs(T, E, K, seed=10)
    idx[3, 1] = idx[3, 0]
    check(z, idx, [0, 17, T], dgate, "same index twice")
    b = Balance(z, idx, [0, T], torch.ones(1), dgate)
    b.idx[5, 0], b.idx[6, 3] = -1, E
    b()
    counts, _, _, dz = b.outputs()
    assert int(counts.sum()) == T * K - 2
    assert bool(dz.isfinite().all())


def test_gradient_against_differences():
    """Central differences of the definition in 64 bits (counts held), along a direction."""
    T, E, K = 50, 12, 3
    z, idx, _ = inputs(T, E, K, seed=11)
    off, dloss = [0, 20, 50], torch.tensor([0.7, -1.3])
    b = Balance(z, idx, off, dloss)
    b()
    dz = b.outputs()[3].double()
    way = torch.randn((T, E), generator=torch.Generator().manual_seed(12), dtype=torch.float64)

    def total(step):
        out, zz = 0.0, z.double() + step * way
        for q in range(2):
            s = torch.sigmoid(zz[off[q]:off[q + 1]])
            share = (s / s.sum(1, keepdim=True)).mean(0)
            n = torch.bincount(idx[off[q]:off[q + 1]].flatten().long(), minlength=E).double()
            out += float(dloss[q]) * float((n * E / (K * len(s)) * share).sum())
        return out
    h = 1e-4
    num = (total(h) - total(-h)) / (2 * h)
    # the differences' own error: h^2/6 of a third derivative of order the gradient's sum
    assert abs(num - float((dz * way).sum())) <= 1e-6 * float((dz * way).abs().sum())


def test_bit_for_bit_and_streams():
    """The same bits on a second run, on another stream, and of two calls at once on two
    streams with workspaces of their own."""
    T, E, K = 5000, 256, 8
    g = torch.Generator().manual_seed(13)
    z = torch.randn((T, E), generator=g)
    idx = torch.rand((T, E), generator=g).topk(K, dim=1).indices.int()
    dgate = torch.randn((T, K), generator=g)
    off, dloss = [0, 999, 3500, T], torch.tensor([1.0, 2.0, 3.0])
    runs = [Balance(z, idx, off, dloss, dgate) for _ in range(3)]
    runs[0]()
    torch.cuda.synchronize()
    a, c = torch.cuda.Stream(), torch.cuda.Stream()
    runs[1](a)
    runs[2](c)
    ref = runs[0].outputs()
    for r in runs[1:]:
        for x, y in zip(ref, r.outputs()):
            assert torch.equal(x, y)


def test_captured_and_replayed():
    """Captured into a graph, replayed with new logits between eager work."""
    T, E, K = 700, 64, 4
    z, idx, dgate = inputs(T, E, K, seed=14)
    off, dloss = [0, 300, 300, T], torch.tensor([1.0, 2.0, 3.0])
    b = Balance(z, idx, off, dloss, dgate)
    b()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b()
    for i in range(4):
        zi, ii, di = inputs(T, E, K, seed=20 + i)
        b.z.copy_(zi)
        b.idx.copy_(ii)
        b.dgate.copy_(di)
        b.gate.copy_(gates(zi, ii))
        b.dz.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        got = b.outputs()
        eager = Balance(zi, ii, off, dloss, di)
        eager()
        for x, y in zip(got, eager.outputs()):
            assert torch.equal(x, y), i


# ---------------- the router's backward for a dense gradient ----------------
def dense(T, H, E, act, seed, scale=1e-3):
    from mixture_experts_layer_added_amd import _lib as L
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if act == "f32" else torch.bfloat16
    x = torch.randn((T, H), generator=g).to(dt)
    w = torch.randn((E, H), generator=g) * 0.02
    dz = torch.randn((T, E), generator=g) * scale
    return run_dense(x, w, dz, act), (x, w, dz), L


def run_dense(x, w, dz, act, stream=None):
    from mixture_experts_layer_added_amd import _lib as L
    (T, H), E = x.shape, w.shape[0]
    p = problem(T, E, 1, H, act)
    n = L.moe_workspace_bytes(p, L.MOE_CALL_ROUTER_BACKWARD_DENSE)
    ws = torch.full((n + 256,), 0x7f, dtype=torch.uint8, device="cuda")
    dx = torch.full((T + 1, H), float("nan"), device="cuda")
    dw = torch.full((E + 1, H), float("nan"), device="cuda")
    L.moe_router_backward_dense(p, x.cuda(), w.cuda(), dz.cuda(), dx, dw, ws, n, stream)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 0x7f).all()) and bool(dx[T:].isnan().all()) and \
        bool(dw[E:].isnan().all()), "a write behind a buffer"
    return dx[:T].cpu(), dw[:E].cpu()


def near(got, a, b):
    ref, mag = a.double() @ b.double(), a.double().abs() @ b.double().abs()
    tol = (a.shape[1] + 16) * 2.0 ** -23
    err = (got.double() - ref).abs()
    assert bool((err <= tol * mag).all()), float((err / mag.clamp(min=1e-300)).max() / tol)
    return float((err / mag.clamp(min=1e-300)).max() * 2 ** 23)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E", [(1, 128, 1), (1, 256, 16), (5, 128, 3), (64, 128, 64),
                                   (127, 384, 48), (129, 128, 100), (300, 640, 256),
                                   (257, 128, 512), (1000, 384, 33), (2100, 256, 72),
                                   (4099, 128, 8)])
def test_dense_router_backward(T, H, E, act):
    (dx, dw), (x, w, dz), _ = dense(T, H, E, act, seed=T + E)
    a = near(dx, dz, w)
    b = near(dw, dz.t(), x)
    log(f"    T={T} H={H} E={E} {act}: dx within {a:.2f}, dw within {b:.2f} of 2^-23 sum |ab|")


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_dense_router_backward_range(act):
    """Gradients from 1e-30 to 1e10 in one matrix, and rows and columns of zeros."""
    T, H, E = 200, 256, 40
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, H), generator=g).to(torch.float32 if act == "f32" else torch.bfloat16)
    w = torch.randn((E, H), generator=g) * 10.0 ** torch.randint(-6, 4, (E, 1), generator=g)
    dz = torch.randn((T, E), generator=g) * 10.0 ** torch.randint(-30, 11, (T, 1), generator=g)
    dz[7] = 0
    dz[:, 5] = 0
    dx, dw = run_dense(x, w, dz, act)
    near(dx, dz, w)
    near(dw, dz.t(), x)
    assert not dx[7].any() and not dw[5].any()


def test_dense_router_backward_repeats():
    """The same bits again, on another stream, and replayed from a graph."""
    from mixture_experts_layer_added_amd import _lib as L
    (dx, dw), (x, w, dz), _ = dense(777, 384, 48, "bf16", seed=2)
    again = run_dense(x, w, dz, "bf16", torch.cuda.Stream())
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    p = problem(777, 48, 1, 384)
    n = L.moe_workspace_bytes(p, L.MOE_CALL_ROUTER_BACKWARD_DENSE)
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
    xd, wd, zd = x.cuda(), w.cuda(), dz.cuda()
    gx, gw = torch.empty((777, 384), device="cuda"), torch.empty((48, 384), device="cuda")
    L.moe_router_backward_dense(p, xd, wd, zd, gx, gw, ws, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        L.moe_router_backward_dense(p, xd, wd, zd, gx, gw, ws, n)
    for i in range(3):
        zd.copy_(dz * (i + 1))
        gx.fill_(float("nan"))
        gw.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ex, ew = run_dense(x, w, dz * (i + 1), "bf16")
        assert torch.equal(gx.cpu(), ex) and torch.equal(gw.cpu(), ew), i
