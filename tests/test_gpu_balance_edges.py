"""The balance loss and its gradient at the edges of their inputs: infinite and NaN logits, rows
of saturated logits with large and small weights, and no token lost or taken twice where chunks
and sequences meet.

Tolerances as in test_gpu_balance.py (u = 2^-24): a share is within 32 u, the gradient within 128 u
of the magnitude that its bracket can cancel from.  A sum of shares adds u for each addition in
its longest chain, here counted from the sum's own structure (see `additions`)."""
import pytest

from test_gpu_balance import Balance, U, inputs, reference

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def up(a, b):
    return -(-a // b)


def additions(T, E, n_seq, length):
    """The longest chain of additions behind a mean share.  A token has 4 to 32 lanes (a count
    that holds for the fewest tokens a wave takes at once, 2, is an upper bound for all).  Up to
    512 tokens: 16 waves side by side, the wave's groups (at most 4 steps), the 16 waves.  More:
    chunks of 16 to 64 tokens up to 65,536 tokens, then as many as make 1024 chunks, 4 waves
    each; then a sequence's chunks over the rows of a workgroup of at least 256 threads (E/4 up to a
    power of two of them a row), and those rows in a tree."""
    if T <= 512:
        return up(length, 16 * 2) + 4 + 16
    chunk = 16
    while chunk * (256 if chunk < 64 else 1024) < T:
        chunk *= 2
    row = 1
    while 4 * row < E:
        row *= 2
    rows = max(256 // row, 1)
    return up(chunk, 4 * 2) + 4 + 2 + up(up(length, chunk) + 1, rows) + 10


def check(z, idx, off, dloss, dgate=None, skip=()):
    """Counts, shares and losses of every sequence but those in `skip`, and their gradients."""
    b = Balance(z, idx, off, dloss, dgate)
    b()
    counts, prob, loss, dz = b.outputs()
    rc, rp, rl, rg, mag = reference(z, idx, off, dloss, dgate)
    assert torch.equal(counts, rc)
    T, E, n = *z.shape, len(off) - 1
    for q in range(n):
        if q in skip:
            continue
        tol = (32 + 3 + additions(T, E, n, off[q + 1] - off[q])) * U
        err = (prob[q].double() - rp[q]).abs()
        assert bool((err <= tol * rp[q]).all()), (q, float((err / rp[q]).max() / U), tol / U)
        assert abs(float(loss[q]) - float(rl[q])) <= (tol + 32 * U) * float(rl[q]), q
    return prob, loss, dz, rg, mag


def near(dz, rg, mag):
    """2^-126 more: a result below the smallest normal number may be flushed."""
    err = (dz.double() - rg).abs()
    assert bool((err <= 128 * U * mag + 2.0 ** -126).all()), float(
        (err / (128 * U * mag + 2.0 ** -126)).max())


@pytest.mark.parametrize("E", [5, 16, 32, 48, 50, 64, 100, 128, 256, 257, 384, 512])
@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("with_gates", [False, True])
def test_infinite_logits(E, T, with_gates):
    """The clamp makes them 80 and -80: a row of -inf has equal shares, as a row of +inf has."""
    K = min(E, 4)
    z, idx, dgate = inputs(T, E, K, seed=E + T)
    z[0] = -INF
    z[3] = INF
    z[4, ::2] = -INF
    z[5, 1::3] = INF
    z[T - 2, 0], z[T - 2, E - 1] = -INF, INF
    z[T - 1] = -INF
    off = [0, 3, 20, T - 1, T]
    dloss = torch.tensor([1.0, -0.5, 2.0, 0.25])
    _, _, dz, rg, mag = check(z, idx, off, dloss, dgate if with_gates else None)
    near(dz, rg, mag)
    assert not dz[0].any() and not dz[3].any() and not dz[T - 1].any()


@pytest.mark.parametrize("E", [5, 16, 32, 50, 64, 128, 256, 257, 384, 512])
@pytest.mark.parametrize("T", [40, 600])
def test_nan_logits(E, T):
    """A NaN logit has a NaN affinity: its sequence's shares and loss and its token's gradient
    are NaN, every other sequence and token as without it."""
    K = min(E, 4)
    z, idx, dgate = inputs(T, E, K, seed=2 * E + T)
    z[25, E // 2] = NAN
    off = [0, 20, 31, T - 3]
    dloss = torch.tensor([1.0, -0.5, 2.0])
    for gates in (None, dgate):
        prob, loss, dz, rg, mag = check(z, idx, off, dloss, gates, skip=(1,))
        assert bool(prob[1].isnan().all()) and bool(loss[1].isnan())
        assert bool(dz[25].isnan().all())
        keep = torch.arange(T) != 25
        near(dz[keep], rg[keep], mag[keep])


@pytest.mark.parametrize("E,K", [(8, 1), (48, 3), (64, 8), (256, 8), (384, 6)])
@pytest.mark.parametrize("weight", [2.0 ** 20, 1.0, 2.0 ** -30])
def test_saturated_rows(E, K, weight):
    """Rows whose logits are all near the lower clamp have affinities of 1e-35 and a sum whose
    reciprocal is 1e34: the gradient, a share times a difference of weights, is an ordinary
    number, whatever the loss's weight."""
    T = 64
    z, idx, dgate = inputs(T, E, K, seed=E)
    z[::2] = z[::2] * 2 - 74
    z[1] = -80.0
    off = [0, 1, 2, 40, T]  # sequences of one token among them
    dloss = torch.tensor([1.0, -1.0, 0.7, -0.3]) * weight
    for gates in (None, dgate * weight * 100):
        _, _, dz, rg, mag = check(z, idx, off, dloss, gates)
        assert bool(dz.isfinite().all())
        near(dz, rg, mag)


def test_padding_behind_a_diverged_sequence():
    """A sequence whose loss has an infinite or NaN gradient keeps it to its own tokens."""
    T, E, K = 90, 64, 4
    z, idx, dgate = inputs(T, E, K, seed=7)
    off = [0, 30, 50, 60]
    for bad in (INF, NAN):
        b = Balance(z, idx, off, torch.tensor([1.0, 1.0, bad]), None)
        b()
        dz = b.outputs()[3]
        assert bool(dz[:50].isfinite().all()) and not dz[60:].any()
        assert not dz[50:60].isfinite().all()
    # several tokens a lane group (from 32,768 tokens on)
    T = 40000
    z, idx = torch.randn((T, E)), torch.zeros((T, 1), dtype=torch.int32)
    b = Balance(z, idx, [0, 11, 1001], torch.tensor([1.0, NAN]), None)
    b()
    dz = b.outputs()[3]
    assert bool(dz[:11].isfinite().all()) and not dz[1001:].any()


@pytest.mark.parametrize("T,E,cuts", [
    (512, 64, [0, 1, 255, 256, 511]),
    (513, 256, [0, 16, 31, 33, 200]),
    (4099, 48, [0, 15, 16, 17, 1000, 1024, 4098]),
    (17001, 64, []),
    (17001, 300, [63, 64, 65, 8191, 8192]),
    (40003, 64, [1, 64, 39000, 39001]),
    (70001, 20, [127, 128, 129, 64000]),
])
def test_every_token_once(T, E, cuts):
    """Shares and losses within the error of their own additions: a token lost or taken twice
    in a sequence of L moves them by about 1/L, 1.5e-5 and more here against under 1e-5."""
    K = 3
    g = torch.Generator().manual_seed(T + E)
    z = torch.randn((T, E), generator=g)
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    off = [0] + cuts + [T]
    check(z, idx, off, torch.ones(len(off) - 1))


@pytest.mark.parametrize("T,E,chunk", [(512, 64, 32), (3000, 64, 16), (6000, 32, 32),
                                       (20000, 256, 64), (20000, 500, 64)])
def test_tokens_at_the_edges(T, E, chunk):
    """One expert that only the first and last tokens of chunks and sequences like: its share is
    theirs alone, so that each of them counts in full."""
    z = torch.randn((T, E), generator=torch.Generator().manual_seed(T))
    z[:, 1] = -30.0
    off = [0, chunk - 1, 5 * chunk, 5 * chunk + 1, 7 * chunk + 3, T - 5]
    edges = {t for o in off for t in (o - 1, o)} | {t for c in range(0, T, chunk)
                                                    for t in (c - 1, c)}
    edges = torch.tensor(sorted(t for t in edges if 0 <= t < T))
    z[edges, 1] = 5.0 + torch.rand(len(edges), generator=torch.Generator().manual_seed(1))
    idx = torch.zeros((T, 2), dtype=torch.int32)
    idx[:, 1] = 1
    check(z, idx, off, torch.ones(len(off) - 1))
