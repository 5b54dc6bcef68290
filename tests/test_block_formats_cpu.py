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


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).double()


def test_the_pairs_that_hold_q():
    # bf16 elements of a row whose largest is scaled into [128, 256): decode,
    # hi + lo / 16; prefill, hi + lo with lo in e5m2.
    m = torch.arange(128, 256, dtype=torch.float64)
    for e in range(0, 40):
        x = m * 2.0 ** -e  # a binade, the largest element's times 2^-e
        hi = _e4m3(x.float())
        off = (x - hi - _e4m3((16 * (x - hi)).float()) / 16).abs().max() / 128
        assert off == 0 if e <= 13 else off <= 2.0 ** -21, e
        off = (x - hi - (x - hi).float().to(torch.float8_e5m2).double()).abs().max() / 128
        assert off == 0 if e <= 13 else off <= 2.0 ** -20, e
