"""NaN and infinities through the E4M3 quantiser, the 8-bit checkpoints and the expert backward
from their codes.

A NaN has a NaN code whatever stands beside it, and the rest of its block is quantised as if it
were not there.  An infinity makes its block's scale infinite: its own code is NaN, the others'
are 0, so every value of the block comes back as NaN (0 times infinity).  No tolerance is needed:
codes and scales are those of the definition, bit for bit (a NaN code's sign aside)."""
import struct

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def blocks(g):
    """name -> 128 values of a block."""
    n = torch.randn((128,), generator=g)

    def with_(base, **at):
        v = base.clone()
        for k, x in at.items():
            v[int(k[1:])] = x
        return v
    zero = torch.zeros(128)
    odd_nan = torch.tensor(struct.unpack("f", b"\xff\xff\xff\xff")[0])
    return {
        "every value NaN": torch.full((128,), NAN),
        "one NaN among zeros": with_(zero, _77=NAN),
        "NaN among values under 2^-90": with_(n * 2.0 ** -100, _0=NAN, _127=-NAN),
        "NaN among ordinary values": with_(n, _3=NAN, _64=NAN),
        "NaN with every bit set": with_(n, _9=odd_nan),
        "NaN among values above 2^100": with_(n * 2.0 ** 110, _31=NAN),
        "all NaN but the largest": with_(torch.full((128,), NAN), _5=-7.5),
        "+inf among ordinary values": with_(n, _8=INF),
        "-inf among zeros": with_(zero, _120=-INF),
        "both infinities": with_(n, _1=INF, _2=-INF),
        "infinity and NaN": with_(n, _40=INF, _41=NAN),
        "every value infinite": torch.full((128,), -INF),
        "no such value": n,
    }


def codes_of(x):
    """The definition along the rows of x [n, 128 k]."""
    w = x.float().view(x.shape[0], -1, 128)
    amax = torch.where(w.isnan(), 0.0, w.abs()).amax(2)
    scale = amax / 448
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (w / scale[:, :, None]).clamp(-448, 448).to(F8).view(torch.uint8)
    return q.view(x.shape[0], -1), scale


def same_codes(got, ref):
    got, ref = got.cpu(), ref.cpu()
    nan = (ref & 0x7f) == 0x7f
    return torch.equal((got & 0x7f) == 0x7f, nan) and torch.equal(got[~nan], ref[~nan])


def matrix(dtype):
    g = torch.Generator().manual_seed(3)
    b = blocks(g)
    names = list(b)
    # every block beside an ordinary one, in rows of 256
    x = torch.cat([torch.stack([b[k] for k in names]), torch.randn((len(b), 128), generator=g)], 1)
    return names, x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", ["rows", "cols", "both"])
def test_quantiser(dtype, form):
    from mixture_experts_layer_added_amd.layer import quantize_fp8
    names, x = matrix(dtype)
    n = len(names)
    ref_q, ref_s = codes_of(x)
    if form != "cols":
        q, s, _, _ = quantize_fp8(x.cuda(), True, form == "both")
        for i, name in enumerate(names):
            assert same_codes(q[i], ref_q[i]), name
            assert torch.equal(s[i].cpu(), ref_s[i]), name
    if form != "rows":  # the blocks down the columns of the transpose
        _, _, qt, st = quantize_fp8(x.t().contiguous().cuda(), form == "both", True)
        for i, name in enumerate(names):
            assert same_codes(qt[i], ref_q[i]), name
            assert torch.equal(st[i].cpu(), ref_s[i]), name
    assert ref_q.shape == (n, 256)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_checkpoint_there_and_back(act):
    from mixture_experts_layer_added_amd import _lib as L
    dt = torch.float32 if act == "f32" else torch.bfloat16
    m = L.MOE_F32 if act == "f32" else L.MOE_BF16
    names, au = matrix(dt)  # rows of [gate | up], I = 128
    R = len(names)
    p = L.problem(R, 128, 4, 1, 1, 1, 1, 128, 0, m, m)
    q = torch.empty((R, 256), dtype=torch.uint8, device="cuda")
    s = torch.empty((R, 2), device="cuda")
    L.moe_checkpoint_save(p, au.cuda(), q, s)
    back, h = torch.empty((R, 256), dtype=dt, device="cuda"), torch.empty((R, 128), dtype=dt,
                                                                          device="cuda")
    L.moe_checkpoint_restore(p, q, s, back, h)
    torch.cuda.synchronize()
    ref_q, ref_s = codes_of(au)
    ref = (ref_q.view(F8).float().view(R, 2, 128) * ref_s[:, :, None]).view(R, 256).to(dt)
    for i, name in enumerate(names):
        assert same_codes(q[i], ref_q[i]) and torch.equal(s[i].cpu(), ref_s[i]), name
        b = back[i].cpu()
        assert torch.equal(b.isnan(), ref[i].isnan()), name
        assert torch.equal(b[~b.isnan()], ref[i][~b.isnan()]), name
        assert torch.equal(h[i].isnan().cpu(), ref[i, :128].isnan()), name
    lost = ~torch.isfinite(au) & torch.isfinite(back.cpu())
    assert not lost.any(), "a value that was not finite came back finite"


def test_expert_backward_from_the_codes():
    """da, du and h of a row whose gate or up block holds such a value: NaN in its columns, and
    the row's dx with them; other rows are those of a batch without it."""
    from mixture_experts_layer_added_amd import _lib as L
    T, H, E, I = 24, 256, 2, 128
    p = L.problem(T, H, E, 1, 1, 1, 1, I, 0, L.MOE_BF16, L.MOE_BF16)
    g = torch.Generator(device="cuda").manual_seed(1)

    def rnd(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()
    w13, w2, dy, au = rnd((E, 2 * I, H), 0.05), rnd((E, H, I), 0.05), rnd((T, H), 1), rnd(
        (T, 2 * I), 1)
    off = torch.tensor([0, 11, T], dtype=torch.int32, device="cuda")
    w13t, w2t = torch.empty_like(w13), torch.empty_like(w2)
    L.moe_pack_expert_weights_transposed(p, w13, w2, w13t, w2t)

    def backward(au):
        q = torch.empty((T, 2 * I), dtype=torch.uint8, device="cuda")
        s = torch.empty((T, 2), device="cuda")
        L.moe_checkpoint_save(p, au, q, s)
        dau, h, dx = torch.empty_like(au), torch.empty_like(au[:, :I]), torch.empty_like(dy)
        h = torch.empty((T, I), dtype=au.dtype, device="cuda")
        L.moe_expert_ffn_backward_input_checkpoint(p, off, w13t, w2t, q, s, dy, dau, h, dx)
        torch.cuda.synchronize()
        return dau.cpu(), h.cpu(), dx.cpu()
    plain = backward(au)
    bad = au.clone()
    bad[5, 70] = NAN           # gate
    bad[17, I + 3] = INF       # up: its block is lost
    got = backward(bad)
    keep = [i for i in range(T) if i not in (5, 17)]
    for a, b in zip(got, plain):
        assert torch.equal(a[keep], b[keep])
    dau, h, dx = got
    assert bool(dau[5, 70].isnan()) and bool(dau[5, I + 70].isnan()) and bool(h[5, 70].isnan())
    assert int(dau[5].isnan().sum()) == 2 and int(h[5].isnan().sum()) == 1
    assert bool(dau[17, :I].isnan().all()) and bool(h[17].isnan().all())
    assert bool(dx[5].isnan().all()) and bool(dx[17].isnan().all())


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_linear_layer(M, bad):
    """A NaN or infinite activation reaches its token's outputs and its column of dw, one in the
    gradient its token's dx and its row of dw; everything else is as without it."""
    from mixture_experts_layer_added_amd.layer import Fp8Linear
    N, K, r = 256, 384, M - 1
    g = torch.Generator(device="cuda").manual_seed(M)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda").bfloat16()
    w, x, dy = rnd(N, K), rnd(M, K), rnd(M, N)

    def step(x, dy):
        lin = Fp8Linear(w, train=True)
        y = lin.forward(x)
        dx = lin.backward(dy)
        torch.cuda.synchronize()
        return y.cpu(), dx.cpu(), lin.dw.cpu()
    y0, dx0, dw0 = step(x, dy)
    rows = torch.arange(M) != r
    xb = x.clone()
    xb[r, 200] = bad
    y, dx, dw = step(xb, dy)
    cols = torch.arange(K) != 200
    assert bool(y[r].isnan().all()) and torch.equal(y[rows], y0[rows])
    assert torch.equal(dx, dx0)
    assert bool(dw[:, 200].isnan().all()) and torch.equal(dw[:, cols], dw0[:, cols])
    db = dy.clone()
    db[r, 70] = bad
    y, dx, dw = step(x, db)
    outs = torch.arange(N) != 70
    assert torch.equal(y, y0)
    assert bool(dx[r].isnan().all()) and torch.equal(dx[rows], dx0[rows])
    assert bool(dw[70].isnan().all()) and torch.equal(dw[outs], dw0[outs])
