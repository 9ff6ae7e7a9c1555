"""quantize_mxfp4 and quantize_fp8 of matrices with one row or one column, whose strides say
nothing: the same codes and scales as for a copy."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def views():
    g = torch.Generator().manual_seed(4)
    x = torch.randn((70, 96), generator=g).cuda().bfloat16()
    yield x[:, :1].contiguous().t()                 # [1, 70], strides (1, 1)
    yield x[0].expand(1, 96)                        # [1, 96], row stride 0
    yield x[3:4, 5:77]                              # a row inside a matrix
    yield x.t()[:, 2:3]                             # [96, 1], strides (1, 96)
    yield x[:, 9:10]                                # [70, 1], strides (96, 1)
    yield x[5:6, 7:8].t()                           # one element


@pytest.mark.parametrize("name", ["quantize_mxfp4", "quantize_fp8"])
@pytest.mark.parametrize("i", range(6))
def test_one_row_or_column(i, name):
    from mixture_experts_layer_added_amd import layer
    x, f = list(views())[i], getattr(layer, name)
    plain = torch.empty(x.shape, dtype=x.dtype, device="cuda").copy_(x)
    a, b = f(x, True, True), f(plain, True, True)
    torch.cuda.synchronize()
    n, m = x.shape
    block = 32 if name == "quantize_mxfp4" else 128
    for got, want, scale in zip(a, b, (False, True, False, True)):
        k = -(-(m if got is a[0] or got is a[1] else n) // block)
        if name == "quantize_mxfp4":
            w = k if scale else 16 * k
        else:
            w = got.shape[1] if scale else (m if got is a[0] else n)
        assert torch.equal(got[:, :w], want[:, :w])


def test_overlapping_rows_are_refused():
    from mixture_experts_layer_added_amd.layer import quantize_mxfp4
    x = torch.zeros((8, 8), device="cuda")
    for bad in (x[0].expand(3, 8), x.t(), x[:, ::2]):
        with pytest.raises(AssertionError):
            quantize_mxfp4(bad)
