"""Windowed decode over a block-scaled cache on the GPU, against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa
import seen_reference as seen

pytestmark = pytest.mark.gpu
DEV = "cuda"

MFA = dict(heads=64, kv_heads=1, dim=256)
GQA = dict(heads=64, kv_heads=4, dim=128)
FIVE = dict(heads=40, kv_heads=8, dim=128)
TWELVE = dict(heads=24, kv_heads=2, dim=256)
SINGLE = dict(heads=3, kv_heads=3, dim=128)


def case(lens, window, sinks, poison=True, **kw):
    c = ref.Case(lens, **kw)
    if poison:   # what no new token sees holds NaN, under table entries outside the pool
        seen.hide(c, lambda b, L: seen.window_seen(L, c.tokens, window, sinks).any(0))
    return c


def decoder(c, window, sinks, lens="plan", **kw):
    host = c.seq_lens.tolist() if lens == "plan" else lens
    return mfa.BlockDecoder(len(c.seq_lens), c.columns, c.pages, num_q_heads=c.heads, num_kv_heads=c.kv_heads,
                            head_dim=c.dim, scale_tokens=c.scale_tokens, tokens_per_seq=c.tokens, host_seq_lens=host,
                            window=window, sinks=sinks, **kw)


def device(c):
    return [x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.block_table, c.seq_lens)]


def expect(c, window, sinks, **kw):
    return seen.decode(c, lambda b, L: seen.window_seen(L, c.tokens, window, sinks), c.tokens, seen.two_e4m3, **kw)


LENS = [1, 2, 63, 64, 65, 0, 127, 128, 129, 200, 517]


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (2, 64), (63, 5), (64, 0), (65, 64), (128, 65), (129, 130), (200, 0),
                                           (1000, 4), (2 ** 31 - 1, 2 ** 31 - 1), (3, 700)])
@pytest.mark.parametrize("shape, block", [(MFA, 64), (GQA, 32), (TWELVE, 16)])
def test_window(shape, block, window, sinks):
    c = case(LENS, window, sinks, **shape, scale_tokens=block, seed=sinks)
    out, lse = decoder(c, window, sinks, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    seen.check(out, lse, expect(c, window, sinks))


@pytest.mark.parametrize("window, sinks", [(1, 0), (2, 1), (3, 0), (62, 63), (64, 64), (130, 1), (300, 67)])
@pytest.mark.parametrize("shape, tokens", [(MFA, 2), (MFA, 4), (GQA, 3), (GQA, 4), (FIVE, 4), (TWELVE, 3), (SINGLE, 2)])
def test_window_of_several_new_tokens(shape, tokens, window, sinks):
    c = case([1, 2, 0, 3, 4, 64, 66, 128, 129, 131, 192, 255, 400], window, sinks, **shape, tokens=tokens, scale_tokens=32, seed=tokens)
    out, lse = decoder(c, window, sinks, flags=mfa.MFA_PLAN_CHECK)(*device(c))
    seen.check(out, lse, expect(c, window, sinks))


@pytest.mark.parametrize("ctas", [0, 1, 2, 5, 17, 64])
@pytest.mark.parametrize("shape, tokens", [(MFA, 1), (GQA, 1), (TWELVE, 3)])
def test_window_split_over_any_grid(shape, tokens, ctas):
    c = case([1700, 0, 129, 1, 2300, 901], 700, 70, **shape, tokens=tokens, scale_tokens=32, seed=ctas)
    out, lse = decoder(c, 700, 70, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    seen.check(out, lse, expect(c, 700, 70))


@pytest.mark.parametrize("way, lens, shape, ctas", [
    ("clusters", [3000] * 20, MFA, 0), ("clusters", [700, 1300], FIVE, 80), ("clusters", [900] * 130, MFA, 0),
    ("even", [9000, 100, 3000], MFA, 0), ("clusters", [5000, 3], SINGLE, 48), ("even", [5000, 3, 3, 3, 3, 3], GQA, 0), ("cost", [700] * 200, SINGLE, 0),
    ("cost", [100, 3000, 700, 0, 1], GQA, 7)])
def test_every_way_to_split_and_lengths_other_than_planned(way, lens, shape, ctas):
    window, sinks = 600, 5
    c = case(lens, window, sinks, poison=False, **shape, scale_tokens=32, seed=ctas)
    dec = decoder(c, window, sinks, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)
    ways = {"cost": 0, "even": mfa.MFA_PLAN_EVEN_SPLIT, "clusters": mfa.MFA_PLAN_UNIT_CLUSTERS}
    assert dec.plan.flags & ~mfa.MFA_PLAN_CHECK == ways[way] | mfa.MFA_PLAN_WINDOW
    d = device(c)
    seen.check(*dec(*d), expect(c, window, sinks))
    c.seq_lens = torch.tensor([min(n, max(1, n * 3 // 5)) for n in lens], dtype=torch.int32)
    seen.check(*dec(*d[:6], c.seq_lens.to(DEV)), expect(c, window, sinks))


def test_a_decode_loop_grows_past_its_plan():
    """A decoder planned for short sequences runs them as they grow, and from a bound alone."""
    window, sinks = 130, 3
    c = case([600, 333], window, sinks, poison=False, **GQA, seed=3)
    d = device(c)
    for dec in (decoder(c, window, sinks, lens=[1, 1], flags=mfa.MFA_PLAN_CHECK), decoder(c, window, sinks, lens=None, flags=mfa.MFA_PLAN_CHECK)):
        for lens in ([1, 1], [64, 200], [131, 64], [600, 333]):
            c.seq_lens = torch.tensor(lens, dtype=torch.int32)
            seen.check(*dec(*d[:6], c.seq_lens.to(DEV)), expect(c, window, sinks))


def test_a_window_over_the_whole_sequence_is_the_decode_without():
    c = ref.Case([5, 700, 1300, 64], **MFA, scale_tokens=16, seed=4)
    d = device(c)
    kw = dict(num_q_heads=64, head_dim=256, scale_tokens=16, host_seq_lens=c.seq_lens.tolist())
    a = mfa.BlockDecoder(4, c.columns, c.pages, **kw)(*d)
    b = mfa.BlockDecoder(4, c.columns, c.pages, window=1300, **kw)(*d)
    want = ref.decode(c)
    for got in (a, b):   # (not the same bits: small elements of q are more exact with a window)
        seen.check(*got, want)
    assert torch.equal(want[0], expect(c, 1300, 0)[0])


def test_long_contexts_and_bad_pages():
    """Only the seen pages' ids are looked at; one outside the pool among them reads as zeros and is reported."""
    rng = np.random.default_rng(1)
    c = case([70001, 3, 40000] + rng.integers(0, 3000, 20).tolist(), 1000, 4, poison=False, heads=8, kv_heads=1, dim=128, seed=4)
    d = device(c)
    dec = decoder(c, 1000, 4, flags=mfa.MFA_PLAN_CHECK)
    seen.check(*dec(*d), expect(c, 1000, 4))
    table = d[5].clone()
    table[0, 5:1000] = 1 << 30      # tokens 320 .. 63999 of the first sequence: not seen
    seen.check(*dec(*d[:5], table, d[6]), expect(c, 1000, 4))
    table[0, 1093] = -5             # its last page
    with pytest.raises(mfa.MfaError) as e:
        dec(*d[:5], table, d[6])
    assert e.value.status == mfa.MFA_ERR_DEVICE_CHECK
    assert mfa.mfa_read_device_status(dec.workspace) == mfa.MFA_DEV_BAD_BLOCK


def test_window_in_a_graph_and_on_another_stream():
    c = case([900, 2000, 77, 0], 300, 10, **GQA, tokens=2, scale_tokens=32, seed=8)
    d, dec, want = device(c), decoder(c, 300, 10), expect(c, 300, 10)
    first = dec(*d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = dec(*d, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = dec(*d)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got in (first, other, held):
        seen.check(*got, want)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
