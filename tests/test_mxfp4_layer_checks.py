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


def mx_weights(n, I, H):
    return [torch.zeros(s, **u8) for s in ((n, 2 * I, H // 2), (n, H, I // 2), (n, 2 * I, H // 32),
                                           (n, H, I // 32))]


def wrong_weights(w):
    """One tensor at a time: a group fewer, half the rows, half the columns, another type."""
    for i, t in enumerate(w):
        for bad in (t[1:], t[:, :t.shape[1] // 2].contiguous(),
                    t[:, :, :t.shape[2] // 2].contiguous(), t.to(torch.int16)):
            yield [*w[:i], bad, *w[i + 1:]]


def test_share_of_mxfp4(Y, MoeError):
    good = mx_weights(3, 128, 256)
    for w in wrong_weights(good):
        with pytest.raises(AssertionError):
            Y.ExpertShare(0, *w, expert="mxfp4")
    with pytest.raises(MoeError, match="host memory"):
        Y.ExpertShare(0, *good, expert="mxfp4")


@pytest.mark.parametrize("expert", ["bf16", "f32"])
def test_share(Y, MoeError, expert):
    dt = torch.float32 if expert == "f32" else torch.bfloat16
    good = [torch.zeros((3, 256, 256), dtype=dt), torch.zeros((3, 256, 128), dtype=dt)]
    turned = [good[0].transpose(1, 2), good[1]]
    for w in [*wrong_weights(good), turned]:
        with pytest.raises(AssertionError):
            Y.ExpertShare(0, *w, expert=expert)
    share = Y.ExpertShare(0, *good, expert=expert)
    with pytest.raises(MoeError, match="host memory"):
        share.forward(torch.zeros((2, 256), dtype=dt), torch.zeros((2, 1), dtype=torch.int32),
                      torch.zeros((2, 1)))


def test_layer_of_mxfp4(Y, MoeError):
    shape = Y.Shape(T=8, H=256, E=2, G=1, M=1, K=1, J=1, I=128, S=1, expert="mxfp4")
    router, bias = torch.zeros((2, 256)), torch.zeros((2,))
    good = mx_weights(3, 128, 256)
    for w in wrong_weights(good):
        with pytest.raises(AssertionError):
            Y.MoELayer(shape, router, bias, *w, device="cpu")
    with pytest.raises(MoeError, match="host memory"):
        Y.MoELayer(shape, router, bias, *good, device="cpu")
