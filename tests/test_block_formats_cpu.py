"""The number formats in which the block-scaled attention kernels hand q and
the probabilities to the tensor core, enumerated (nothing here reaches a GPU)."""
import torch


def _e5m2(x):
    """The e5m2 value nearest to an f16, saturating."""
    return x.clamp(-57344, 57344).to(torch.float8_e5m2).to(torch.float16)


def _three(p):
    """a + b / 8 + c / 64 of f16 values, the differences in f16."""
    a = _e5m2(p)
    r = (p - a) * 8
    b = _e5m2(r)
    c = _e5m2((r - b) * 8)
    return a.double() + b.double() / 8 + c.double() / 64


def test_three_e5m2_numbers_hold_an_f16():
    p = torch.arange(0x7800, dtype=torch.int16).view(torch.float16)  # 0 .. below 2^15
    off = (_three(p) - p.double()).abs()
    assert p.max() < 2 ** 15 and off.max() <= 2.0 ** -23
    assert (off[p > 2.0 ** -12 * 1.01] == 0).all()


def test_a_probability_keeps_eleven_bits_far_below_the_largest():
    # P of the largest weight lies in [2^11, 2^15)
    gen = torch.Generator().manual_seed(1)
    x = torch.exp2(torch.rand(1 << 20, generator=gen, dtype=torch.float64) * 45 - 30).float()
    off = (_three(x.half()) - x.double()).abs()
    big = x >= 2.0 ** -11
    assert (off[big] <= 2.0 ** -11 * x[big].double()).all()
    assert off[~big].max() <= 2.0 ** -33 * 2.0 ** 11
