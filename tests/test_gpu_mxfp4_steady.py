"""The MXFP4 product and the experts past their start-up: every ring of the kernels goes round more
than once, sums are split over k in every tile, and there are more groups than lanes.

Tolerances as in test_gpu_mxfp4: exact products, (blocks + 8) 2^-23 of sum |a b| for the fp32 sums,
half a step of bf16."""
import pytest

from mxfp4_cases import up, values
from test_gpu_mxfp4 import check_experts, check_product, groups, product, run_experts

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def codes(n, cols, g, low=121, high=133):
    """Random codes and scales [low, high) of [n, cols]; what lies behind the last block is NaN."""
    kb = up(cols, 32) // 32
    q = torch.randint(0, 256, (n, 16 * kb), generator=g, dtype=torch.uint8)
    s = torch.full((n, up(kb, 16)), 255, dtype=torch.uint8)
    s[:, :kb] = torch.randint(low, high, (n, kb), generator=g, dtype=torch.uint8)
    return q, s


# M, N, K and the parts that k is cut into.  The tile that each of them is made for: rows and columns
PRODUCTS = [
    (1, 70, 9001, 1), (1, 70, 16384, 1), (16, 50, 9001, 1), (32, 33, 9001, 1), (32, 70, 16384, 1),
    (46, 56, 6163, 1),                                     # 32 x 32
    (130, 2100, 4500, 1), (300, 300, 12000, 8),            # 64 x 64
    (600, 2100, 4500, 1), (1539, 130, 11535, 6),           # 128 x 64
    (1200, 2100, 4500, 1), (65, 2898, 13219, 9),           # 128 x 128
    (2500, 2900, 4500, 1), (711, 2771, 13622, 3),          # 128 x 256
    (3000, 4200, 4500, 1), (1685, 2518, 10594, 3)]         # 256 x 256


@pytest.mark.parametrize("out", ["bf16", "f32", "add"])
@pytest.mark.parametrize("M,N,K,parts", PRODUCTS)
def test_product(M, N, K, parts, out):
    from mixture_experts_layer_added_amd import _lib as L
    assert L.moe_gemm_mxfp4_workspace_bytes(M, N, K) == (parts * M * up(N, 4) * 4 if parts > 1 else 0)
    g = torch.Generator().manual_seed(M + N + K)
    a, b = codes(M, K, g), codes(N, K, g)
    c0 = torch.randn((M, N), generator=g) * 1000 if out == "add" else None
    c = product(a, b, M, N, K, "bf16" if out == "bf16" else "f32", c0=c0)
    rows = torch.unique(torch.cat([torch.arange(0, M, max(1, M // 40)),
                                   torch.arange(max(0, M - 5), M)]))
    check_product(c[rows], values(a[0][rows], a[1][rows], K), values(*b, K),
                  None if c0 is None else c0[rows])


def run_codes(T, H, I, counts, seed):
    """As run_experts, with random codes in place of quantised numbers."""
    from mixture_experts_layer_added_amd import _lib as L
    g = torch.Generator().manual_seed(seed)
    NG = len(counts)
    off, token = groups(counts, T, 0, seed)
    K = -(-off[-1] // T)
    p = L.problem(T, H, NG, 1, 1, K, 1, I, 0, L.MOE_BF16, L.MOE_MXFP4)
    R = off[-1] + 3
    xq, xs = codes(T, H, g, 124, 127)
    w = []
    for rows, cols in ((2 * I, H), (H, I)):
        q = torch.randint(0, 256, (NG, rows, cols // 2), generator=g, dtype=torch.uint8)
        w.append((q, torch.randint(118, 121, (NG, rows, cols // 32), generator=g, dtype=torch.uint8)))
    (q13, s13), (q2, s2) = w
    p13 = torch.empty((L.moe_mxfp4_packed_bytes(NG, 2 * I, H),), dtype=torch.uint8, device="cuda")
    p2 = torch.empty((L.moe_mxfp4_packed_bytes(NG, H, I),), dtype=torch.uint8, device="cuda")
    dev = [t.cuda() for t in (q13, s13, q2, s2, xq, xs)]
    L.moe_pack_expert_weights_mxfp4(p, *dev[:4], p13, p2)
    hq = torch.full((R, I // 2), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((R, up(I // 32, 16)), 0x55, dtype=torch.uint8, device="cuda")
    y = torch.full((R, H), 5.0, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    tok = torch.cat([token, torch.full((3,), -5)]).to(torch.int32).cuda()
    L.moe_expert_ffn_up_mxfp4(p, dev[4], dev[5], xs.shape[1], tok, offs, p13, hq, hs, hs.shape[1])
    L.moe_expert_ffn_down_mxfp4(p, hq, hs, hs.shape[1], offs, p2, y)
    torch.cuda.synchronize()
    return dict(off=off, token=token, X=values(xq, xs, H), hq=hq.cpu(), hs=hs.cpu(), y=y.cpu(),
                W13=[values(a, b, H) for a, b in zip(q13, s13)],
                W2=[values(a, b, I) for a, b in zip(q2, s2)])


@pytest.mark.parametrize("T,H,I,counts", [
    (200, 2048, 2048, [33, 65, 97, 128, 129, 300]), (150, 3968, 2176, [64, 96, 1, 130, 256]),
    (90, 1664, 3968, [32, 128, 160, 0, 70])])
def test_experts_long_rows(T, H, I, counts):
    """Row tiles of 32, 64, 96 and 128 rows, a group's only one and not, over many steps of k; even and
    odd numbers of 128 of k."""
    check_experts(run_codes(T, H, I, counts, T), H, I)


def many(NG, kind):
    g = torch.Generator().manual_seed(NG)
    c = torch.randint(0, 4, (NG,), generator=g)
    if kind == "gaps":  # none around the borders of 64 groups
        for b in range(0, NG + 1, 64):
            c[max(0, b - 3):b + 3] = 0
    elif kind == "last":
        c[:] = 0
    c[-1], c[NG // 2] = 140, 33
    if kind == "borders":
        c[63::64], c[64::64] = 130, 5
    return c.tolist()


@pytest.mark.parametrize("kind", ["any", "gaps", "last", "borders"])
@pytest.mark.parametrize("NG", [65, 130, 257, 513])
def test_experts_in_many_groups(NG, kind):
    counts = many(NG, kind)
    T = max(40, up(sum(counts), 12) // 12)
    check_experts(run_experts(T, 256, 128, counts, seed=NG, S=1 if NG % 2 else 0), 256, 128)


# ---------------------------------------------------------------------------
# zeros against the largest scale, NaN in bf16
# ---------------------------------------------------------------------------
FORMS = [(3, 50), (20, 50), (40, 40), (150, 200), (1200, 2100)]


@pytest.mark.parametrize("K", [320, 301])
@pytest.mark.parametrize("M,N", FORMS)
def test_zeros_times_the_largest_scale(M, N, K):
    """Codes 0 of a against codes under E = 254, whose values are infinite in fp32 from code 4 on,
    add nothing; codes past K neither, whatever their scale."""
    g = torch.Generator().manual_seed(M + K)
    a, b = codes(M, K, g), codes(N, K, g)
    last = up(K, 32) // 32 - 1
    for block in (2, last):  # with K = 301 the last one's codes past K stay as they are
        n = min(32, K - 32 * block)
        part = a[0][:, 16 * block:16 * block + 16]
        keep = torch.arange(32).view(16, 2) >= n
        mask = (keep[:, 0] * 0x0f + keep[:, 1] * 0xf0).to(torch.uint8)
        part &= mask
        b[1][:, block] = 254
    c = product(a, b, M, N, K, "f32")
    A, B = values(*a, K), values(*b, K)
    assert bool(c.isfinite().all())
    rows = torch.arange(0, M, max(1, M // 50))
    check_product(c[rows], A[rows], B)


@pytest.mark.parametrize("M,N", FORMS)
def test_nan_in_bf16(M, N):
    g = torch.Generator().manual_seed(M)
    a, b = codes(M, 320, g), codes(N, 320, g)
    a[1][1, 3], b[1][7, 0] = 255, 255
    c = product(a, b, M, N, 320, "bf16")
    want = torch.zeros((M, N), dtype=torch.bool)
    want[1], want[:, 7] = True, True
    assert torch.equal(c.isnan(), want)


def test_experts_zeros_times_the_largest_scale():
    """Tokens whose last 128 columns are zero, weights of the quantiser's largest scale there."""
    T, H, I = 50, 384, 128
    g = torch.Generator().manual_seed(6)
    x = torch.randn((T, H), generator=g)
    x[:, H - 128:] = 0
    w = [(torch.randn((2 * I, H), generator=g) * 0.1, torch.randn((H, I), generator=g) * 0.1)
         for _ in range(2)]
    plain = run_experts(T, H, I, [40, 30], seed=2, x=x, w=w)
    for w13, _ in w:
        w13[:, H - 128:] = 3e38
    large = run_experts(T, H, I, [40, 30], seed=2, x=x, w=w)
    for k in ("hq", "hs", "y"):
        assert torch.equal(plain[k], large[k])
