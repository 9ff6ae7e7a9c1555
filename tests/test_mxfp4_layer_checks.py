"""What the helpers and layers of MXFP4 and of a share refuse before they touch a device: shapes and
types that do not fit together, which would have a kernel read past a tensor.  Host tensors suffice:
where shapes fit, they reach the binding, which refuses host memory."""
import pytest

torch = pytest.importorskip("torch")
u8 = dict(dtype=torch.uint8)


@pytest.fixture(scope="module")
def Y():
    from mixture_experts_layer_added_amd import layer
    return layer


@pytest.fixture(scope="module")
def MoeError():
    from mixture_experts_layer_added_amd import MoeError
    return MoeError


def test_dequantize(Y, MoeError):
    q, s = torch.zeros((6, 64), **u8), torch.zeros((6, 16), **u8)
    for a, b in ((q, s[:5]), (q[:5], s), (q[None], s[None]), (q, s[0]), (q.float(), s),
                 (q, s.float())):
        with pytest.raises(AssertionError):
            Y.dequantize_mxfp4(a, b, 100)
    with pytest.raises(MoeError, match="host memory"):
        Y.dequantize_mxfp4(q, s, 100)
