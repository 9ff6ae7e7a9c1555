"""Stochastic rounding of bf16 to MXFP4, which goes through a conversion instruction with a seed: every
finite bf16 inside the range of every scale that the quantiser gives, with every random byte, against
the definition, bit for bit.  Along the rows, along the columns, and along the rows where both forms
are written.  (The definition in 64 bits on the GPU: powers of two by their bits, so each step of it is
exact.)"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_layer_added_amd import _lib
    _lib.lib()


def definition(x, r, scale):
    """Codes 0 .. 15 of bf16 x under scale code `scale`, rounded by the bytes r."""
    power = torch.tensor((127 - scale + 1023) << 52, device=DEV).view(torch.float64)
    a = x.double().abs() * power
    part = (a >= 2).long() + (a >= 4).long()  # steps of 1/2, 1, 2
    f = torch.where(part == 0, 2 * a, torch.where(part == 1, a, 0.5 * a))
    low = f.floor()
    up = (f - low) * 256 > r.double() + 0.5
    return low.long() + up.long() + 2 * part | torch.signbit(x).long() << 3


def numbers(scale):
    """Every finite bf16 in the scale's range, 31 a row, behind each row one that fixes the scale."""
    top = (scale + 2) << 7 | 0x40 if scale < 253 else 0x7f7f  # 6 times the scale, or the last number
    bits = torch.arange(top + 1, device=DEV)
    bits = torch.cat([bits, bits | 0x8000])
    bits = torch.cat([bits, bits.new_zeros(-len(bits) % 31)]).view(-1, 31)
    bits = torch.cat([bits, torch.full_like(bits[:, :1], top)], 1)
    return bits.to(torch.int16).view(torch.bfloat16)


def unpack(q):
    return torch.stack([q & 15, q >> 4], -1).flatten(1).long()


@pytest.mark.parametrize("first", range(0, 254, 32))
def test_every_number_scale_and_byte(first):
    from mixture_experts_layer_added_amd.layer import quantize_mxfp4
    for scale in range(first, min(first + 32, 254)):
        x = numbers(scale)
        n = len(x)
        r = torch.arange(256, device=DEV).to(torch.uint8).repeat_interleave(n)[:, None]
        r = r.expand(-1, 32).contiguous()
        x = x.repeat(256, 1)
        want = definition(x, r, scale)
        q, s, _, _ = quantize_mxfp4(x, True, False, r)
        q2, s2, _, _ = quantize_mxfp4(x, True, True, r)
        _, _, q3, s3 = quantize_mxfp4(x.t().contiguous(), False, True, r.t().contiguous())
        for codes, scales in ((q, s), (q2, s2), (q3, s3)):
            assert bool((scales[:, 0] == scale).all()), scale
            bad = unpack(codes) != want
            assert not bool(bad.any()), (scale, x[bad][:4], r[bad][:4], unpack(codes)[bad][:4],
                                         want[bad][:4])
