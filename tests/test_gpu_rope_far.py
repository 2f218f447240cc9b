"""Rotary positions as far as 32 bits go, on the GPU, against decimal arithmetic of 60 digits."""
import decimal
import math

import pytest
import torch

import decode_attention_02_gb300 as mfa
from test_rope_table import exact_turns

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scale", [1.0, 16.0, 0.3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_positions_have_the_angles_of_their_exact_products(scale, dtype):
    """The angle: 2^-31 of a turn, and half a step of its fp32 half turns (2^-25 of one); cos and sin of it to two
    steps of theirs: 2^-21 in all, and half a step of the output type."""
    pairs = 64
    rope = mfa.Rope(2 * pairs, (pairs,), position_scale=scale)
    where = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -1234567890, 131072, 1]
    x = torch.zeros((len(where), 1, 2 * pairs), dtype=dtype)
    x[..., :pairs] = 1.0
    out, _ = rope(x.to(DEV), None, torch.tensor([where], dtype=torch.int32, device=DEV))
    back, _ = rope(x.to(DEV), None, torch.tensor([where], dtype=torch.int32, device=DEV), inverse=True)
    turns = exact_turns((pairs,), 0, 1e4, scale)
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        for r, p in enumerate(where):
            for i in range(pairs):
                a = 2 * math.pi * float((turns[i] * p) % 1)
                for got, want in ((out[r, 0, i], math.cos(a)), (out[r, 0, i + pairs], math.sin(a)),
                                  (back[r, 0, i + pairs], -math.sin(a))):
                    assert abs(float(got) - want) <= 2.0 ** -21 + torch.finfo(dtype).eps / 2, (p, i)
