"""Decode over a block-scaled cache where one token outweighs thousands of others, on the GPU.

Such rows (a first token with half of the weight and more) are made of many weights that are each next
to nothing beside the largest: bounds on the output, not on one weight at a time.
"""
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa
from test_gpu_block import DEV, FIVE, GQA, MFA, TWELVE, check, decoder, device

pytestmark = pytest.mark.gpu

PAGE = 64
# A weight is rounded to f16 and to two e4m3 parts: 2^-10 and 2^-8 of itself.
WEIGHT = 2.0 ** -8 + 2.0 ** -10


def put(c, name, b, x):
    """Store sequence b's rows x [tokens, kv_heads, dim], each block under its least power-of-two scale."""
    cache, scale = getattr(c, name + "_cache"), getattr(c, name + "_scale")
    n, block = x.shape[0], c.scale_tokens
    for t in range(0, n, block):
        page, slot = int(c.block_table[b, t // PAGE]), t % PAGE
        rows = x[t:t + block].transpose(0, 1)                                    # [kv_heads, rows, dim]
        s = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)).clamp(min=2.0 ** -100) / 448)))
        scale[page, :, slot // block] = s
        cache[page, :, slot:slot + rows.shape[1]] = (rows / s[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def sinks(lens, shape, tokens, nats, at, deviation, mean, sink_value, seed):
    """Scores: normal, `deviation` wide; `nats` more for token `at` (or several).  Values: normal about `mean`,
    token `at`'s `sink_value` times that."""
    c = ref.Case(lens, **shape, tokens=tokens, scale_tokens=16, seed=seed, poison=False)
    gen = torch.Generator().manual_seed(seed + 1)
    c.q[..., 0] = 128.0
    at = torch.as_tensor(at).reshape(-1)
    for b, n in enumerate(lens):
        k = torch.randn((n, c.kv_heads, c.dim), generator=gen) * deviation
        k[..., 0] = 0.0
        k[at, :, 0] = nats * c.dim ** 0.5 / 128.0
        v = torch.randn((n, c.kv_heads, c.dim), generator=gen) + mean
        v[at] *= sink_value
        put(c, "k", b, k)
        put(c, "v", b, v)
    return c


def check_norms(c, out, bound):
    want = ref.decode(c)[0]
    off = (out.cpu().double() - want).norm(dim=-1) / want.norm(dim=-1).clamp(min=1e-300)
    assert float(off.max()) <= bound, (float(off.max()), bound)


# Each weight is off by WEIGHT of itself at most, in the mean square by less than half of that; the
# tile of a token that outweighs it is held to 2^-21 of that token's weight a token (half a step of the
# second part, 2^-15, where the largest is at least 2^6).
@pytest.mark.parametrize("length, nats, mean, deviation", [
    (4096, 8.8, 0.0, 1.0), (4096, 10.2, 0.0, 1.0), (16384, 10.2, 0.0, 1.0), (32768, 10.9, 0.5, 1.0), (32768, 12.0, 0.5, 0.5)])
@pytest.mark.parametrize("ctas", [1, 0])
def test_a_first_token_of_small_value_does_not_drown_the_others(length, nats, mean, deviation, ctas):
    c = sinks([length], dict(heads=16, kv_heads=1, dim=256), 1, nats, 0, deviation, mean, 0.02, seed=length)
    out, _ = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    check_norms(c, out, 2.0 ** -7)


@pytest.mark.parametrize("shape, tokens", [(MFA, 1), (MFA, 2), (GQA, 1), (GQA, 4), (FIVE, 2), (TWELVE, 3)])
def test_first_tokens_of_small_value_in_every_layout(shape, tokens):
    c = sinks([4100, 3000], shape, tokens, 9.5, 0, 1.0, 0.25, 0.02, seed=tokens)
    for ctas in (2, 0):
        out, _ = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
        check_norms(c, out, 2.0 ** -7)


@pytest.mark.parametrize("nats", [4.0, 5.5, 7.0, 8.0, 9.0, 11.0, 14.0])
@pytest.mark.parametrize("at", [[0], [0, 40], [70, 71, 3], [700, 740]])
def test_a_few_tokens_of_small_value_however_far_above(nats, at):
    """From the same range as the others to far above all of them, in one and several quarters of a tile."""
    c = sinks([8000], dict(heads=16, kv_heads=1, dim=256), 1, nats, at, 1.0, 0.0, 0.02, seed=17)
    out, _ = decoder(c, force_ctas=1, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    check_norms(c, out, 2.0 ** -7)


@pytest.mark.parametrize("at", [[8060, 8070], [500, 600, 700], [0, 130, 1024]])
def test_tokens_of_small_value_in_neighbouring_tiles(at):
    """Each tile's other tokens keep their share: 4 % of the row's norm a tile, where they were lost."""
    c = sinks([15000], dict(heads=32, kv_heads=1, dim=256), 1, 11.2, at, 0.3, 0.0, 0.0, seed=3)
    for ctas in (1, 2):
        out, _ = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
        check_norms(c, out, 2.0 ** -7)


@pytest.mark.parametrize("length", [4096, 65536])
@pytest.mark.parametrize("nats", [7.0, 9.9, 12.0, 14.1, 16.0, 20.0])
@pytest.mark.parametrize("at", [0, 1001])
def test_the_weights_of_many_equal_tokens_add_up(length, nats, at):
    """All values one: the row is one; and the outweighing token's zero: what the others have together."""
    shape = dict(heads=8, kv_heads=1, dim=128)
    for sink_value in (1.0, 0.0):
        c = ref.Case([length], **shape, scale_tokens=64, seed=1, poison=False)
        c.q[..., 0] = 128.0
        k = torch.zeros((length, 1, 128))
        k[at, :, 0] = nats * 128 ** 0.5 / 128.0
        v = torch.ones((length, 1, 128))
        v[at] = sink_value
        put(c, "k", 0, k)
        put(c, "v", 0, v)
        want, want_lse, _, lse_tol = ref.decode(c)
        largest = float(torch.exp(float(c.rows("k", 0, length)[0][0, at, 0]) * 128 / 128 ** 0.5 - want_lse).max())
        tol = WEIGHT * want + 127 * 2.0 ** -21 * largest + 2.0 ** -18
        for ctas in (1, 0):
            out, lse = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
            off = (out.cpu().double() - want).abs() - tol
            assert bool((off <= 0).all()), (ctas, sink_value, float(off.max()), float(tol.max()))
            assert bool(((lse.cpu().double() - want_lse).abs() <= lse_tol).all())


def test_peaks_that_come_and_go():
    """Every 700 tokens one that outweighs the rest by 2^20, the others of small value: references fall and rise."""
    length = 9001
    c = ref.Case([length], heads=64, kv_heads=1, dim=256, scale_tokens=16, seed=4, poison=False)
    gen = torch.Generator().manual_seed(5)
    c.q[..., 0] = 128.0
    k = torch.randn((length, 1, 256), generator=gen)
    k[..., 0] = 0.0
    k[300::700, :, 0] = 14.0 / 8
    v = torch.randn((length, 1, 256), generator=gen)
    put(c, "k", 0, k)
    put(c, "v", 0, v)
    for ctas in (1, 3, 0):
        out, lse = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
        check(c, out, lse)
        check_norms(c, out, 2.0 ** -7)


@pytest.mark.parametrize("rise", [122, 105, -30, -41])
@pytest.mark.parametrize("shape, tokens", [(MFA, 1), (GQA, 2)])
def test_value_scales_near_the_ends_of_their_range(shape, tokens, rise):
    """All value scales 2^rise times an ordinary one: sums and lse keep every weight."""
    c = ref.Case([700, 90], **shape, tokens=tokens, scale_tokens=32, seed=rise + 200, poison=False)
    c.v_scale *= 2.0 ** rise
    for ctas in (2, 0):
        out, lse = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
        check(c, out, lse)
