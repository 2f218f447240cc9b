"""The table of rotary frequencies against decimal arithmetic of 60 digits (no GPU)."""
import ctypes
import decimal

import pytest

import block_reference as ref
import decode_attention_02_gb300 as mfa
from decode_attention_02_gb300 import build

D = decimal.Decimal
PI = D("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return mfa.load_library()


def exact_turns(sections, flags, theta, scale):
    """Turns a position of each pair, as decimals (theta and scale are the doubles that the call gets)."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        log_theta, seen, out = D(theta).ln(), [0] * len(sections), []
        for i, a in enumerate(ref.rope_axes(sections, bool(flags & mfa.MFA_ROPE_INTERLEAVED))):
            power = D(seen[a]) / sections[a] if flags & mfa.MFA_ROPE_OWN_SPECTRUM else D(i) / sum(sections)
            seen[a] += 1
            out.append((-power * log_theta).exp() * D(scale) / (2 * PI))
        return out


@pytest.mark.parametrize("sections, flags", [((64,), 0), ((128,), 0), ((22, 21, 21), 0), ((24, 20, 20), mfa.MFA_ROPE_INTERLEAVED),
                                             ((8, 0, 3, 5), mfa.MFA_ROPE_INTERLEAVED | mfa.MFA_ROPE_OWN_SPECTRUM),
                                             ((1, 30), mfa.MFA_ROPE_OWN_SPECTRUM), ((1,), 0), ((256,), 0)])
@pytest.mark.parametrize("theta", [1.0, 1.0 + 2.0 ** -52, 2.0, 1e4, 5e5, 1e6 / 3, 1e300])
@pytest.mark.parametrize("scale", [1.0, 16.0, 0.1, 1e-300])
def test_every_fraction_is_the_nearest(sections, flags, theta, scale):
    full = (list(sections) + [0] * 4)[:4]
    table = mfa.mfa_rope_table(mfa.MfaRopeConfig(512, 2 * sum(sections), len(sections), (ctypes.c_int32 * 4)(*full), 0, flags,
                                                 theta, scale))
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        for i, (x, turns) in enumerate(zip(table, exact_turns(sections, flags, theta, scale))):
            off = (D(x.turns) - turns * 2 ** 64) % 2 ** 64        # (sign of the dividend)
            off = min(abs(off), 2 ** 64 - abs(off))
            assert off <= D("0.5000001"), (i, x.turns, off)
