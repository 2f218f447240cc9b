"""The rounding of a tree decode's weights that include/mfa.h states, from the arithmetic of its two parts (no GPU)."""
import torch


def split(P):
    """A weight times its value scale, relative to its row's reference: f16, then an e4m3 part and an e5m2 one of the rest."""
    f = P.half().float()
    hi = f.to(torch.float8_e4m3fn).float()
    return hi.double() + (f - hi).to(torch.float8_e5m2).double()


def stated(P, largest):
    """What a weight may be off by, with the largest of the 128 tokens about it."""
    largest = torch.as_tensor(largest, dtype=P.dtype)
    small = torch.minimum(torch.maximum(2.0 ** -3 * P, 2.0 ** -14 * largest), 2.0 ** -11 * largest)
    return torch.where(P >= 2.0 ** -4 * largest, 2.0 ** -7 * P, small)


def test_two_parts_hold_what_is_stated():
    """A tile's largest P lies between 2^-2, under which references fall, and 2^8.75, over which they rise."""
    for top in (-2.0, -1.5, 0.0, 4.0, 8.75):
        P = torch.exp2(torch.linspace(top - 30, top, 400001, dtype=torch.float64)).float()
        off = (split(P) - P.double()).abs()
        assert bool((off <= stated(P.double(), 2.0 ** top)).all()), top
    # and they hold no more than half of it: what vanishes, or is rounded to the smallest step
    P = torch.tensor([2.0 ** -17])
    assert float((split(P) - P.double()).abs()) == 2.0 ** -15 * 2.0 ** -2
