"""A share of the experts: pairs sorted by expert, rows sent there and back with their weights, and
the gradients, against the definitions.

Tolerances: the sorting is exact, a row sent with its weight is one rounded product (fp32: 2^-24 of
it, bf16: that and 2^-8).  A sum of K products in fp32: K 2^-24 sum |w v|, rounded once more.  A
dot over H: every partial sum rounded, H 2^-24 sum |x v|."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def want_sort(idx, first, count):
    T, K = idx.shape
    e = idx.flatten().long() - first
    here = ((e >= 0) & (e < count)).nonzero().flatten()
    pair = here[e[here].sort(stable=True).indices]
    row = torch.full((T * K,), -1, dtype=torch.int32)
    row[pair] = torch.arange(len(pair), dtype=torch.int32)
    off = torch.zeros((count + 1,), dtype=torch.int32)
    off[1:] = torch.bincount(e[here], minlength=count).cumsum(0)
    return off, (pair // K).to(torch.int32), row.view(T, K)


def sort(idx, first, count, stream=None):
    from mixture_experts_layer_added_amd import _lib as L
    T, K = idx.shape
    off = torch.full((count + 1,), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((T * K,), -9, dtype=torch.int32, device="cuda")
    row = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    n = L.moe_sort_by_expert_workspace_bytes(T, K, count)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    L.moe_sort_by_expert(T, K, idx.cuda() if idx.numel() else None, first, count, off, tok, row, ws,
                         n, stream)
    return off, tok, row


@pytest.mark.parametrize("T,K,E,first,count", [
    (1, 1, 1, 0, 1), (1, 8, 256, 0, 256), (3, 2, 8, 5, 2), (64, 8, 256, 32, 32), (128, 8, 64, 0, 64),
    (129, 8, 64, 60, 4), (1024, 1, 512, 0, 512), (1025, 1, 9, 0, 9), (2000, 5, 48, 40, 8),
    (50000, 8, 256, 0, 256), (40000, 16, 512, 500, 12), (300, 4, 16, 20, 4)])
def test_sort(T, K, E, first, count):
    g = torch.Generator().manual_seed(T + count)
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)  # an expert may come twice
    off, tok, row = sort(idx, first, count)
    torch.cuda.synchronize()
    w_off, w_tok, w_row = want_sort(idx, first, count)
    assert torch.equal(off.cpu(), w_off) and torch.equal(row.cpu(), w_row)
    n = int(w_off[-1])
    assert torch.equal(tok.cpu()[:n], w_tok) and bool((tok[n:] == -9).all())


@pytest.mark.parametrize("T", [100, 5000])
def test_sort_any_index(T):
    """Indices of any value; every choice the same expert; none of them here."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    idx = torch.tensor([lo, -1, 0, 3, 4, 5, hi, 7], dtype=torch.int32).repeat(T, 1)
    for first, count in ((3, 2), (0, 512), (hi - 1, 2), (5, 1), (6, 1)):
        off, tok, row = sort(idx, first, count)
        torch.cuda.synchronize()
        w_off, w_tok, w_row = want_sort(idx, first, count)
        assert torch.equal(off.cpu(), w_off) and torch.equal(row.cpu(), w_row)
        assert torch.equal(tok.cpu()[:len(w_tok)], w_tok)
    same = torch.full((T, 8), 3, dtype=torch.int32)
    off, tok, row = sort(same, 2, 3)
    torch.cuda.synchronize()
    assert off.tolist() == [0, 0, 8 * T, 8 * T]
    assert torch.equal(row.cpu().flatten(), torch.arange(8 * T, dtype=torch.int32))


def test_no_tokens():
    from mixture_experts_layer_added_amd import _lib as L
    off, _, _ = sort(torch.empty((0, 8), dtype=torch.int32), 0, 300)
    for f in (L.moe_dispatch, L.moe_collect):
        f(L.MOE_BF16, 0, 8, 128, None, 128, None, None, None, 128)
    for f in (L.moe_dispatch_backward, L.moe_collect_backward):
        f(L.MOE_F32, 0, 8, 128, None, 128, None, None, None, 128, None, 128)
    torch.cuda.synchronize()
    assert off.tolist() == [0] * 301


def strided(T, H, ld, dtype, g, fill=None):
    t = torch.randn((T, ld), generator=g).to(dtype)
    if fill is not None:
        t[:, :] = fill
    return t


CASES = [(1, 1, 1, 0), (3, 2, 7, 1), (5, 8, 128, 0), (9, 4, 2000, 8), (17, 16, 2049, 0),
         (40, 6, 4096, 16), (2, 3, 7168, 0), (33, 8, 500, 12)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("T,K,H,pad", CASES)
def test_there_and_back(T, K, H, pad, dtype, weights):
    from mixture_experts_layer_added_amd import _lib as L
    g = torch.Generator().manual_seed(T * 7 + H)
    dt, code, ld = DT[dtype], L.MOE_F32 if dtype == "f32" else L.MOE_BF16, H + pad
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    idx = torch.randint(0, 5, (T, K), generator=g, dtype=torch.int32)
    off, tok, row = sort(idx, 1, 3)
    torch.cuda.synchronize()
    n, R = int(off[-1]), T * K
    r = row.cpu().long()
    x, ys = strided(T, H, ld, dt, g), strided(R, H, ld, dt, g)
    ys[n:] = float("nan")  # rows of no pair: not used
    w = torch.randn((T, K), generator=g) if weights else None
    wd = w.cuda() if weights else None
    xc, yc = x.cuda(), ys.cuda()
    rows = torch.full((R, ld), 5.0, dtype=dt, device="cuda")
    back = torch.full((T, ld), 5.0, dtype=dt, device="cuda")
    L.moe_dispatch(code, T, K, H, xc, ld, row, wd, rows, ld)
    L.moe_collect(code, T, K, H, yc, ld, row, wd, back, ld)
    rows2, back2 = torch.full_like(rows, 5.0), torch.full_like(back, 5.0)
    dw = torch.full((2, T, K), 5.0, device="cuda") if weights else [None, None]
    L.moe_dispatch_backward(code, T, K, H, yc, ld, row, wd, xc if weights else None, ld, back2, ld,
                            dw[0])
    L.moe_collect_backward(code, T, K, H, xc, ld, row, wd, yc if weights else None, ld, rows2, ld,
                           dw[1])
    torch.cuda.synchronize()
    # both ways move the same rows, with dots or without
    assert torch.equal(rows, rows2) and torch.equal(back, back2)
    rows, back = rows.cpu().double(), back.cpu().double()
    assert bool((rows[n:] == 5).all() and (rows[:, H:] == 5).all() and (back[:, H:] == 5).all())
    X, Y = x[:, :H].double(), ys[:, :H].double()
    W = w.double() if weights else torch.ones((T, K), dtype=torch.float64)
    sums, size = torch.zeros((T, H), dtype=torch.float64), torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            if r[t, k] < 0:
                if weights:
                    assert dw[0][t, k] == 0 and dw[1][t, k] == 0
                continue
            v, one = Y[r[t, k]], W[t, k] * X[t]
            assert bool(((rows[r[t, k], :H] - one).abs() <= (half + 2.0 ** -23) * one.abs()).all())
            sums[t] += W[t, k] * v
            size[t] += (W[t, k] * v).abs()
            if weights:
                dot, most = (X[t] * v).sum(), (X[t] * v).abs().sum()
                for i in (0, 1):
                    assert abs(dw[i][t, k].item() - dot) <= H * 2.0 ** -24 * most
    err = (back[:, :H] - sums).abs()
    assert bool((err <= (K + 1) * 2.0 ** -24 * size + half * sums.abs() * (1 + 2.0 ** -8)).all())


def test_gradients_by_differences():
    """dispatch_backward and collect_backward against differences of the forward calls (fp32; the
    calls are linear in each of their arguments)."""
    from mixture_experts_layer_added_amd import _lib as L
    g = torch.Generator().manual_seed(4)
    T, K, H = 6, 3, 40
    idx = torch.randint(0, 6, (T, K), generator=g, dtype=torch.int32)
    _, _, row = sort(idx, 1, 4)
    R = T * K
    x, w = torch.randn((T, H), generator=g).cuda(), torch.randn((T, K), generator=g).cuda()
    up_r, up_t = torch.randn((R, H), generator=g).cuda(), torch.randn((T, H), generator=g).cuda()
    ys = torch.randn((R, H), generator=g).cuda()

    def there(x, w):
        o = torch.zeros((R, H), device="cuda")
        L.moe_dispatch(L.MOE_F32, T, K, H, x, H, row, w, o, H)
        return (o.double() * up_r.double()).sum()

    def back(ys, w):
        o = torch.empty((T, H), device="cuda")
        L.moe_collect(L.MOE_F32, T, K, H, ys, H, row, w, o, H)
        return (o.double() * up_t.double()).sum()

    dx, dw = torch.empty_like(x), torch.empty_like(w)
    L.moe_dispatch_backward(L.MOE_F32, T, K, H, up_r, H, row, w, x, H, dx, H, dw)
    dys, dw2 = torch.zeros_like(ys), torch.empty_like(w)
    L.moe_collect_backward(L.MOE_F32, T, K, H, up_t, H, row, w, ys, H, dys, H, dw2)
    for f, a, b, da, db in ((there, x, w, dx, dw), (back, ys, w, dys, dw2)):
        for i, (v, d) in enumerate(((a, da), (b, db))):
            way = torch.randn(v.shape, generator=g).cuda()
            args = [[a, b], [a, b]]
            args[0][i], args[1][i] = v + way, v - way
            slope = (f(*args[0]) - f(*args[1])) / 2
            want = (d.double() * way.double()).sum()
            # sums of up to 720 terms of order 1, each off by a few 2^-24
            assert abs(slope - want) <= 720 * 8 * 2.0 ** -24 * 10


def test_streams_and_graph():
    """On another stream, and captured with the sort and replayed on new choices."""
    from mixture_experts_layer_added_amd import _lib as L
    g = torch.Generator().manual_seed(8)
    T, K, H, E = 700, 4, 96, 24
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32).cuda()
    x, w = torch.randn((T, H), generator=g).cuda(), torch.rand((T, K), generator=g).cuda()
    off = torch.empty((9,), dtype=torch.int32, device="cuda")
    tok = torch.zeros((T * K,), dtype=torch.int32, device="cuda")
    row = torch.empty((T, K), dtype=torch.int32, device="cuda")
    n = L.moe_sort_by_expert_workspace_bytes(T, K, 8)
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
    xs, y = torch.zeros((T * K, H), device="cuda"), torch.empty((T, H), device="cuda")

    def step():
        L.moe_sort_by_expert(T, K, idx, 8, 8, off, tok, row, ws, n)
        L.moe_dispatch(L.MOE_F32, T, K, H, x, H, row, None, xs, H)
        L.moe_collect(L.MOE_F32, T, K, H, xs, H, row, w, y, H)

    def want():
        here = (idx >= 8) & (idx < 16)
        return x.double() * (w.double() * here).sum(1, keepdim=True)

    def check():
        assert bool(((y.double() - want()).abs() <= 8 * 2.0 ** -24 * x.abs().double() * K).all())

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        idx.copy_(torch.randint(0, E, (T, K), generator=g, dtype=torch.int32))
        x.copy_(torch.randn((T, H), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        check()
