"""The router's backward for a dense logit gradient where the sizes of its operands go against
each other, and at its finest: an error counted against the terms of each sum, whatever else
stands in the row or column.

Tolerance: fp32 operands in three bf16 parts (8, 8 and 8 bits; what is left is under 2^-27 of the
value) and the products of the parts down to 2^-18 of the term: what is left out is 2 2^-27 for
the operands' rests and 2 2^-27 for the products of second and third parts, 2^-25 in all.  Each
addition is rounded or truncated, 2^-23 of the running sum at most; the products of small parts
come first and are far below it.  One term: (1 + 1/4 + 1/64) 2^-23, taken as 1.5 2^-23; n terms:
(n + 16) 2^-23 of sum |a b|, as in test_gpu_balance.py."""
import pytest

from gpu_cases import log
from test_gpu_balance import near, run_dense

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E", [(70, 256, 8), (70, 128, 64), (1100, 128, 100), (300, 4096, 40)])
@pytest.mark.parametrize("spread", [20, 30, 40])
def test_large_gradients_meet_small_weights(T, H, E, act, spread):
    """Expert e has gradients of 2^-a_e and weights of 2^(a_e - spread): every term of a sum is
    as large as the others, while each row of dz and each column of W_r spans 2^spread."""
    g = torch.Generator().manual_seed(E + spread)
    a = torch.linspace(0, spread, E).round()
    a = a[torch.randperm(E, generator=g)]
    x = torch.randn((T, H), generator=g).to(torch.float32 if act == "f32" else torch.bfloat16)
    dz = torch.randn((T, E), generator=g) * torch.exp2(-a)
    w = torch.randn((E, H), generator=g) * torch.exp2(a - spread)[:, None]
    dx, dw = run_dense(x, w, dz, act)
    e = near(dx, dz, w)
    near(dw, dz.t(), x)
    log(f"    T={T} H={H} E={E} {act} spread 2^{spread}: dx within {e:.2f} of 2^-23 sum |ab|")


def test_one_term():
    """With one expert a result is one product of two fp32 numbers, in dx, and with one token in
    dW."""
    g = torch.Generator().manual_seed(4)
    T, H = 130, 256
    x = torch.randn((T, H), generator=g)
    dz = torch.randn((T, 1), generator=g) * 10.0 ** torch.randint(-12, 12, (T, 1), generator=g)
    w = torch.randn((1, H), generator=g) * 10.0 ** torch.randint(-12, 12, (1, H), generator=g)
    dx, _ = run_dense(x, w, dz, "f32")
    ref = dz.double() @ w.double()
    assert bool(((dx.double() - ref).abs() <= 1.5 * 2.0 ** -23 * ref.abs()).all())
    dz = torch.randn((1, 9), generator=g)
    _, dw = run_dense(x[:1], torch.randn((9, H), generator=g), dz, "f32")
    ref = dz.double().t() @ x[:1].double()
    assert bool(((dw.double() - ref).abs() <= 1.5 * 2.0 ** -23 * ref.abs()).all())


def test_largest_and_smallest_numbers():
    """Operands at the ends of the exponent range, and a product that reaches back to 1."""
    T, H, E = 40, 128, 20
    g = torch.Generator().manual_seed(5)
    big = 3.4e38  # above bf16's largest number, 3.39e38
    x = torch.randn((T, H), generator=g)
    w = torch.randn((E, H), generator=g)
    dz = torch.zeros((T, E))
    dz[0, 3], w[3] = big, w[3] * 1e-38
    dz[1, 4] = -big
    w[4] = w[4] * 1e-3
    dz[2] = torch.randn((E,), generator=g) * 1e-30
    x[1:] *= 1e-3
    x[0] *= 1e-2
    dx, dw = run_dense(x, w, dz, "f32")
    # parts below 2^-133 are rounded to bf16's subnormal step: half of it times the other operand
    ref, mag = dz.double() @ w.double(), dz.double().abs() @ w.double().abs()
    floor = 2.0 ** -134 * (dz.double().abs().sum(1, keepdim=True) +
                           w.double().abs().sum(0, keepdim=True)) + 2.0 ** -126
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())
    assert bool(((dx.double() - ref).abs() <= (E + 16) * 2.0 ** -23 * mag + floor).all())
    near(dw, dz.t(), x)


@pytest.mark.parametrize("T,H,E", [(33, 128, 16), (200, 256, 70)])
def test_non_finite_gradients(T, H, E):
    """A NaN or infinite gradient makes its token's dx and its expert's dW not finite, and
    nothing else."""
    import struct
    g = torch.Generator().manual_seed(6)
    x = torch.randn((T, H), generator=g).bfloat16()
    w = torch.randn((E, H), generator=g)
    odd = torch.tensor(struct.unpack("f", b"\xff\xff\xff\xff")[0])
    for bad in (torch.tensor(float("nan")), torch.tensor(float("inf")), odd):
        dz = torch.randn((T, E), generator=g)
        clean = run_dense(x, w, dz, "bf16")
        dz[9, 5] = bad
        dx, dw = run_dense(x, w, dz, "bf16")
        assert not dx[9].isfinite().any() and not dw[5].isfinite().any()
        rows, experts = torch.arange(T) != 9, torch.arange(E) != 5
        assert torch.equal(dx[rows], clean[0][rows])
        assert torch.equal(dw[experts], clean[1][experts])
