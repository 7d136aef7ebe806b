"""What the gated feed-forward's stash holds of G and U: their upper 24 bits, rounded to nearest, half of the last place off
at most.  Gradients in bf16 do not show which way the last bits go, so the stash itself is read: with the same G and U
everywhere every element of its planes (16 bits of all of G, of all of U, then 8 bits of each) is the same."""
import numpy as np
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu


def parts(v):
    """v as a sum of bf16 numbers, the sum of which fp32 holds exactly."""
    out, left = [], float(v)
    for _ in range(8):
        p = torch.tensor(left, dtype=torch.float64).to(torch.bfloat16)
        if torch.isinf(p):  # (the numbers above bf16's last one)
            p = torch.tensor(3.3895313892515355e38, dtype=torch.float64).to(torch.bfloat16) * np.sign(left)
        out.append(p)
        left -= float(p)
    assert left == 0
    return torch.stack(out)


def kept(m, f, g, u):
    x = torch.ones(m, 8, dtype=torch.bfloat16, device="cuda")
    wg, wu = (parts(v).expand(f, 8).contiguous().cuda() for v in (g, u))
    stash = binding.ffn_stash(x, wg)
    stash.fill_(0)
    binding.ffn_forward(x, wg, wu, stash=stash)
    n, raw = -(-m // 128) * 128 * f, stash.cpu().numpy()
    assert raw.size == 6 * n
    hi, lo = raw[:4 * n].view("<u2").astype(np.uint32), raw[4 * n:].astype(np.uint32)
    values = []
    for which in range(2):
        h, b = hi[which * n:][:n], lo[which * n:][:n]
        assert (np.sort(h)[-m * f:] == h.max()).all() and set(np.unique(h)) <= {0, h.max()}
        values.append(np.array([h.max() << 16 | b.max() << 8], dtype=np.uint32).view(np.float32)[0])
    return [float(v) for v in values]


def f32(bits):
    return float(np.array([bits], dtype=np.uint32).view(np.float32)[0])


# low bits below, at and above half of the last kept place, a carry through all of them, either sign; one row tile and many
BITS = [0x3f800000, 0x3f80007f, 0x3f800081, 0x3f8000ff, 0x3f8012c0, 0x3fffff90, 0x3fffffff, 0x40490fdb, 0x0c812ff0, 0x7e967ec3]


@pytest.mark.parametrize("m,f", [(3, 8), (1100, 2568)])
@pytest.mark.parametrize("at", range(len(BITS)))
def test_rounded_to_nearest(m, f, at):
    g, u = f32(BITS[at]), f32(BITS[-1 - at] | 0x80000000)
    for value, got in zip((g, u), kept(m, f, g, u)):
        place = 2.0 ** (np.floor(np.log2(abs(value))) - 15)  # of 24 bits 15 are the fraction's
        assert abs(got - value) <= place / 2 + abs(value) * 2.0 ** -22, (value, got)  # (the product's own fp32 sum)


def test_the_greatest_number_stays_finite():
    most = f32(0x7f7fffff)
    g, u = kept(3, 8, most, -most)
    assert np.isfinite([g, u]).all() and abs(g / most - 1) <= 2.0 ** -15 and u == -g
