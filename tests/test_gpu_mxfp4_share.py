"""ExpertShare with MXFP4 experts at the ends of its range.  Exact: a token's rows do not depend on
the other tokens of the call."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


@pytest.mark.parametrize("T,K,H,count", [(130, 16, 256, 2), (4104, 16, 65536, 2)])
def test_all_tokens_at_once_and_in_halves(T, K, H, count):
    """More choices than experts; in the second case T*K*H/2 passes 2^31, T*H/2 does not."""
    from mixture_experts_layer_added_amd.layer import ExpertShare, quantize_weights_mxfp4
    g = torch.Generator(device="cuda").manual_seed(T)
    I = 128

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()
    (a, sa), (b, sb) = (quantize_weights_mxfp4(rnd(count, 2 * I, H) / 64),
                        quantize_weights_mxfp4(rnd(count, H, I)))
    share = ExpertShare(3, a, b, sa, sb, "mxfp4")
    x = rnd(T, H)
    idx = torch.randint(0, 40, (T, K), generator=g, device="cuda", dtype=torch.int32)
    gate = torch.rand((T, K), generator=g, device="cuda")
    y = share.forward(x, idx, gate)
    half = T // 2
    parts = [share.forward(x[r].contiguous(), idx[r].contiguous(), gate[r].contiguous())
             for r in (slice(0, half), slice(half, T))]
    torch.cuda.synchronize()
    here = ((idx >= 3) & (idx < 3 + count)).any(1)
    assert bool(y[here].any(1).all()) and not bool(y[~here].any())
    assert torch.equal(y, torch.cat(parts))


def test_sort_of_no_tokens_without_workspace():
    from mixture_experts_layer_added_amd import _lib as L
    off = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    L.moe_sort_by_expert(0, 4, None, 0, 8, off, None, None, None, 0)
    assert off.tolist() == [0] * 9


@pytest.mark.parametrize("expert", ["bf16", "f32"])
def test_training_step_captured(expert):
    """Forward and backward of a share in a graph, replayed on new tokens, choices and gradients, with
    eager steps of another share of the same weights in between: the same bits."""
    from mixture_experts_layer_added_amd.layer import ExpertShare
    g = torch.Generator().manual_seed(11)
    T, K, E, H, I, count = 70, 3, 10, 256, 128, 4
    dt = torch.float32 if expert == "f32" else torch.bfloat16

    def rnd(*shape):
        return torch.randn(shape, generator=g).to(dt).cuda()
    w13, w2 = rnd(count, 2 * I, H) * 0.05, rnd(count, H, I) * 0.05
    share, eager = (ExpertShare(3, w13, w2, expert=expert, train=True) for _ in range(2))
    x, dy = rnd(T, H), rnd(T, H)
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32).cuda()
    gate = torch.rand((T, K), generator=g).cuda()

    def step(s):
        y = s.forward(x, idx, gate)
        return y, *s.backward(dy)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(share)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(share)
    for n in (E, 5, 2 ** 20, E):  # half of the choices here, most, none
        x.copy_(torch.randn(x.shape, generator=g))
        dy.copy_(torch.randn(dy.shape, generator=g))
        idx.copy_(torch.randint(0, n, idx.shape, generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, share.dw13, share.dw2)]
        want = [*step(eager), eager.dw13, eager.dw2]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
