"""MXFP4 and the share of the experts where offsets pass 32 bits, and on two streams at once.

Everything here is exact: the quantisation and the values against their definition, moved rows
against copies, a product of two blocks of ones against its sum, and streams against the same calls
one after the other (no call's result depends on the order of atomics)."""
import pytest

import mxfp4_cases as C

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
FAR = 2 ** 30 + 64  # elements between rows: the third begins past 2^31


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def far(rows, cols, dtype, stride=FAR):
    """[rows, cols] with `stride` elements between rows."""
    t = torch.empty(((rows - 1) * stride + cols,), dtype=dtype, device="cuda")
    return t.as_strided((rows, cols), (stride, 1))


def test_quantize_and_values_far():
    from mixture_experts_layer_added_amd import _lib as L
    from mixture_experts_layer_added_amd import layer as Y
    x = far(4, 100, torch.bfloat16)
    x.copy_(torch.randn(4, 100, generator=torch.Generator().manual_seed(1)))
    q, s, qt, st = Y.quantize_mxfp4(x, True, True)
    for got, scale, src in ((q, s, x), (qt, st, x.t())):
        w_q, w_s = C.quantize(src.cpu())
        assert torch.equal(got.cpu(), w_q) and torch.equal(scale[:, :w_s.shape[1]].cpu(), w_s)
    out = far(4, 100, torch.bfloat16)
    L.moe_dequantize_mxfp4(4, 100, q, q.shape[1], s, s.shape[1], out.data_ptr(), FAR, L.MOE_BF16)
    assert torch.equal(out.cpu().double(), C.values(q, s, 100))


@pytest.mark.parametrize("M", [3, 40])
def test_product_far(M):
    """Two blocks of ones a row: C = 64 everywhere."""
    from mixture_experts_layer_added_amd import _lib as L
    N, K, stride = 40, 64, FAR if M == 3 else 2 ** 26
    ops = []
    for n in (M, N):
        q, s = C.buffers(n, K, 0, 0, "cuda")
        q[:, :32], s[:, :2] = 0x22, 127
        ops += [q, q.shape[1], s, s.shape[1]]
    out = far(M, N, torch.float32, stride)
    n = L.moe_gemm_mxfp4_workspace_bytes(M, N, K)
    assert n == 0
    L.moe_gemm_mxfp4(M, N, K, *ops, out.data_ptr(), stride, L.MOE_F32, 0, None, 0)
    assert bool((out == 64.0).all())


def test_rows_far():
    from mixture_experts_layer_added_amd import _lib as L
    T, K, H = 2, 2, 40
    g = torch.Generator().manual_seed(2)
    row = torch.tensor([[3, 0], [-1, 2]], dtype=torch.int32, device="cuda")
    x, xs = far(T, H, torch.bfloat16), far(T * K, H, torch.bfloat16)
    x.copy_(torch.randn(T, H, generator=g))
    L.moe_dispatch(L.MOE_BF16, T, K, H, x.data_ptr(), FAR, row, None, xs.data_ptr(), FAR)
    for r, t in ((3, 0), (0, 0), (2, 1)):
        assert torch.equal(xs[r], x[t])
    y = far(T, H, torch.bfloat16)
    w = torch.tensor([[1.0, 0.0], [5.0, 2.0]], device="cuda")
    L.moe_collect(L.MOE_BF16, T, K, H, xs.data_ptr(), FAR, row, w, y.data_ptr(), FAR)
    assert torch.equal(y[0], x[0]) and torch.equal(y[1], 2 * x[1])


def test_two_streams_at_once():
    from mixture_experts_layer_added_amd import layer as Y
    g = torch.Generator().manual_seed(3)

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()
    jobs = []
    for i, (T, K, first) in enumerate(((700, 4, 0), (300, 2, 3))):
        H, I, n = 256, 384, 5
        w13, s13 = Y.quantize_weights_mxfp4(rnd(n, 2 * I, H))
        w2, s2 = Y.quantize_weights_mxfp4(rnd(n, H, I))
        share = Y.ExpertShare(first, w13, w2, s13, s2, "mxfp4")
        lin = Y.Fp4Linear(rnd(H, H), train=True, stochastic=False)
        x, dy = rnd(T, H), rnd(T, H)
        idx = torch.randint(0, 8, (T, K), generator=g, dtype=torch.int32).cuda()
        gate = torch.rand(T, K, generator=g).cuda()

        def job(share=share, lin=lin, x=x, dy=dy, idx=idx, gate=gate):
            lin.zero_grad()
            y = share.forward(lin.forward(x), idx, gate)
            return y, lin.backward(dy), lin.dw.clone()
        jobs.append(job)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        got = []
        for s, job in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append([job() for _ in range(3)])
        torch.cuda.synchronize()
        for runs, w in zip(got, want):
            for out in runs:
                assert all(torch.equal(a, b) for a, b in zip(out, w))
