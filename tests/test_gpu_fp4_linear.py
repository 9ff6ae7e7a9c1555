"""Fp4Linear without tokens: empty outputs, weight gradients left as they were.  Exact."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


@pytest.mark.parametrize("stochastic", [False, True])
def test_no_tokens(stochastic):
    from mixture_experts_layer_added_amd.layer import Fp4Linear
    g = torch.Generator().manual_seed(1)
    N, K = 96, 160
    lin = Fp4Linear(torch.randn((N, K), generator=g).bfloat16().cuda(), True, stochastic)
    x, dy = torch.randn((9, K), generator=g).bfloat16().cuda(), torch.randn((9, N), generator=g)
    dy = dy.bfloat16().cuda()
    r = torch.randint(0, 256, dy.shape, generator=g, dtype=torch.uint8).cuda()
    y = lin.forward(x)
    dx = lin.backward(dy, r)
    dw = lin.dw.clone()
    assert bool(dw.any())
    none = lin.forward(x[:0])
    assert none.shape == (0, N) and none.dtype == torch.bfloat16 and none.is_cuda
    back = lin.backward(dy[:0])
    assert back.shape == (0, K) and back.dtype == torch.bfloat16 and back.is_cuda
    with pytest.raises(AssertionError):
        lin.backward(dy)  # of another number of tokens than the last forward's
    torch.cuda.synchronize()
    assert torch.equal(lin.dw, dw)
    lin.zero_grad()
    assert torch.equal(lin.forward(x), y) and torch.equal(lin.backward(dy, r), dx)
    torch.cuda.synchronize()
    assert torch.equal(lin.dw, dw)
    assert Fp4Linear(torch.zeros((N, K), device="cuda").bfloat16()).forward(x[:0]).shape == (0, N)
