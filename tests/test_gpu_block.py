"""Block-scaled 8-bit cache on the GPU: decode and append against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa

pytestmark = pytest.mark.gpu
DEV = "cuda"

MFA = dict(heads=64, kv_heads=1, dim=256)
GQA = dict(heads=64, kv_heads=4, dim=128)
FIVE = dict(heads=40, kv_heads=8, dim=128)      # five query heads a key head
TWELVE = dict(heads=24, kv_heads=2, dim=256)
SINGLE = dict(heads=3, kv_heads=3, dim=128)     # one query head a key head


def decoder(c, lens="plan", **kw):
    host = c.seq_lens.tolist() if lens == "plan" else lens
    return mfa.BlockDecoder(len(c.seq_lens), c.columns, c.pages, num_q_heads=c.heads, num_kv_heads=c.kv_heads,
                            head_dim=c.dim, scale_tokens=c.scale_tokens, tokens_per_seq=c.tokens, host_seq_lens=host,
                            **kw)


def device(c):
    return [x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.block_table, c.seq_lens)]


def check(c, out, lse, expect=None):
    """out (bf16: half a step, 2^-8 of the value, more) and lse within the derived bounds."""
    want, want_lse, tol, lse_tol = expect or ref.decode(c)
    got = out.cpu().double()
    if out.dtype is torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got - want).abs() - tol).max()))
    gl = lse.cpu().double()
    empty = torch.isinf(want_lse)
    assert torch.equal(gl[empty], want_lse[empty])
    off = (gl - want_lse).abs()[~empty]
    assert bool((off <= lse_tol[~empty]).all()), float((off - lse_tol[~empty]).max())
    assert bool((got.reshape(lse.shape + (-1,))[empty] == 0).all())


@pytest.mark.parametrize("shape, block", [(MFA, 64), (MFA, 16), (GQA, 32), (GQA, 64), (FIVE, 16), (TWELVE, 32), (SINGLE, 64)])
@pytest.mark.parametrize("lens", [[1], [64], [63, 65, 127, 128, 129], [0, 5, 0, 300, 1], [0, 0], [517, 2, 1100]])
def test_decode(shape, block, lens):
    c = ref.Case(lens, **shape, scale_tokens=block, seed=len(lens))
    out, lse = decoder(c, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    check(c, out, lse)


@pytest.mark.parametrize("shape", [MFA, GQA, FIVE, TWELVE, SINGLE])
@pytest.mark.parametrize("tokens", [2, 3, 4])
def test_decode_of_several_new_tokens(shape, tokens):
    # shorter than the new tokens (rows that see nothing), across page and tile borders
    c = ref.Case([1, 2, 0, 3, 64, 66, 128, 129, 130, 131, 400], **shape, tokens=tokens, seed=tokens)
    out, lse = decoder(c, flags=mfa.MFA_PLAN_CHECK)(*device(c))
    check(c, out, lse)


@pytest.mark.parametrize("ctas", [1, 2, 5, 17, 64])
@pytest.mark.parametrize("shape, tokens", [(MFA, 1), (GQA, 1), (TWELVE, 3)])
def test_decode_split_over_any_grid(shape, tokens, ctas):
    c = ref.Case([700, 0, 129, 1, 1300], **shape, tokens=tokens, scale_tokens=32, seed=ctas)
    out, lse = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    check(c, out, lse)


WAYS = {"cost": 0, "even": mfa.MFA_PLAN_EVEN_SPLIT, "clusters": mfa.MFA_PLAN_UNIT_CLUSTERS}


@pytest.mark.parametrize("way, lens, shape, kw, ctas", [
    ("clusters", [300] * 130, MFA, dict(), 0),                       # whole units
    ("clusters", [700] * 16, GQA, dict(tokens=2), 0),                # two CTAs a unit
    ("clusters", [700, 129], GQA, dict(tokens=2), 24),               # three; a sequence of two tiles on them
    ("clusters", [1024] * 20, MFA, dict(), 0),                       # four
    ("clusters", [700, 1300], FIVE, dict(), 80),
    ("clusters", [700, 129], GQA, dict(tokens=2), 48),               # six CTAs to six tiles
    ("clusters", [1100] * 8, TWELVE, dict(tokens=3), 112),           # five: five groups of rows
    ("clusters", [900] * 10, MFA, dict(), 0),                        # eight
    ("clusters", [5000, 4990], SINGLE, dict(), 48),                  # eight for one group of rows
    ("even", [900, 1, 0, 200], MFA, dict(), 4),
    ("even", [900, 1, 0, 200], MFA, dict(tokens=3), 12),
    ("even", [1300, 100], GQA, dict(), 16),
    ("even", [1300, 100], TWELVE, dict(tokens=2), 12),
    ("even", [700, 257], MFA, dict(), 10),
    ("even", [700, 129, 2000], FIVE, dict(), 24 * 4),
    ("even", [5000, 3], SINGLE, dict(), 48),
    ("even", [9000, 100, 3000], MFA, dict(), 0),
    ("even", [9000, 100, 0, 3000], GQA, dict(tokens=2), 0),
    ("even", [20000], SINGLE, dict(), 0),
    ("even", [30000], MFA, dict(), 240),                             # more parts than weights held at a time
    ("even", [30000] + [1] * 40, MFA, dict(), 280),
    ("even", [30000] + [1] * 60, GQA, dict(), 1200),
    ("cost", [700] * 200, SINGLE, dict(), 0),
    ("cost", [100, 3000, 700, 0, 1], GQA, dict(), 7),
])
def test_every_way_to_split(way, lens, shape, kw, ctas):
    """Also with device lengths other than those of the plan, as far as it has room for them."""
    c = ref.Case(lens, **shape, **kw, scale_tokens=32, seed=len(lens) + ctas)
    dec = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)
    assert dec.plan.flags & ~mfa.MFA_PLAN_CHECK == WAYS[way]
    d = device(c)
    check(c, *dec(*d))
    c.seq_lens = torch.tensor([max(n // 2, 1) for n in reversed(sorted(lens))][::-1], dtype=torch.int32)
    c.seq_lens = torch.minimum(c.seq_lens, torch.tensor(lens, dtype=torch.int32))
    check(c, *dec(*d[:6], c.seq_lens.to(DEV)))


@pytest.mark.parametrize("kw", [dict(spread=12.0), dict(spread=6.0, pow2=False), dict(q_spread=10.0), dict(pow2=False)])
@pytest.mark.parametrize("shape", [MFA, GQA])
def test_decode_of_scales_and_heads_far_apart(shape, kw):
    """Scales of any positive size, not powers of two alone, and heads of very different norms."""
    c = ref.Case([333, 1024], **shape, scale_tokens=16, seed=3, **kw)
    c.k_scale /= 2.0 ** kw.get("spread", 0.0)     # scores of an ordinary size from the largest keys
    c.q = (c.q.float() / 2.0 ** kw.get("q_spread", 0.0)).bfloat16()
    out, lse = decoder(c, force_ctas=3, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    check(c, out, lse)


@pytest.mark.parametrize("shape, tokens, lens", [(MFA, 2, [33, 200]), (GQA, 3, [34, 129, 66]), (TWELVE, 4, [35, 65]), (FIVE, 1, [300])])
@pytest.mark.parametrize("rise", [20, -20, 60])
def test_a_value_scale_far_from_the_others_costs_no_other_token_its_precision(shape, tokens, lens, rise):
    """The last block's scale 2^rise times what it was: the new tokens that see none of it, and the weights of the
    tokens before it, keep theirs."""
    c = ref.Case(lens, **shape, tokens=tokens, scale_tokens=32, seed=rise + 100, poison=False)
    for b, L in enumerate(lens):
        page, block = int(c.block_table[b, (L - 1) // 64]), (L - 1) % 64 // 32
        c.v_scale[page, :, block] *= 2.0 ** rise
    out, lse = decoder(c, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    check(c, out, lse)


@pytest.mark.parametrize("shape", [MFA, GQA])
def test_blocks_of_zero_values_stay_in_the_sums(shape):
    """As the append leaves them: zero codes under the smallest scale; in front, between others and alone."""
    c = ref.Case([512, 700, 128, 40], **shape, scale_tokens=32, seed=9, poison=False)
    for b, blocks in enumerate(([0, 1, 2, 3, 4, 5, 6], [3, 4, 9, 20], [0, 1, 2, 3], [1])):
        for k in blocks:
            page, at = int(c.block_table[b, k // 2]), k % 2
            c.v_cache[page, :, 32 * at:32 * at + 32] = 0
            c.v_scale[page, :, at] = 2.0 ** -126
    for ctas in (2, 0):
        out, lse = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
        check(c, out, lse)


def test_decode_of_peaked_and_growing_scores():
    """Scores that climb along the sequence (the reference of the weights moves often) and one token that
    outweighs all others."""
    c = ref.Case([900, 640], **MFA, scale_tokens=16, seed=8)
    c.q = (c.q.float() * 4).bfloat16()
    for b in range(2):
        for t in range(0, int(c.seq_lens[b]), 16):
            page = c.block_table[b, t // 64]
            c.k_scale[page, 0, t % 64 // 16] *= 1.0 + t / 200.0
    out, lse = decoder(c, force_ctas=2, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)(*device(c))
    check(c, out, lse)


def test_decode_of_a_long_sequence():
    c = ref.Case([70001, 3], heads=8, kv_heads=1, dim=128, seed=4, poison=False)
    out, lse = decoder(c, flags=mfa.MFA_PLAN_CHECK)(*device(c))
    check(c, out, lse)


def test_decode_of_many_short_sequences():
    """More units than a grid of one CTA per SM has room for, lengths of zero among them."""
    rng = np.random.default_rng(5)
    c = ref.Case(rng.integers(0, 4, 700).tolist(), heads=16, kv_heads=8, dim=128, columns=1, seed=6)
    for kw in (dict(), dict(force_ctas=40)):
        out, lse = decoder(c, flags=mfa.MFA_PLAN_CHECK, **kw)(*device(c))
        check(c, out, lse)


def test_a_table_so_wide_that_costs_pass_32_bits():
    c = ref.Case([700, 0, 129, 1, 1300], **GQA, seed=8)
    q, k, v, ks, vs, table, lens = device(c)
    wide = torch.zeros((5, 15_000_000), dtype=torch.int32, device=DEV)
    wide[:, :c.columns] = table
    dec = mfa.BlockDecoder(5, wide.shape[1], c.pages, num_q_heads=c.heads, num_kv_heads=c.kv_heads, head_dim=c.dim,
                           scale_tokens=c.scale_tokens, host_seq_lens=c.seq_lens.tolist(), force_ctas=7,
                           flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)
    assert dec.plan.flags == mfa.MFA_PLAN_CHECK   # by cost
    check(c, *dec(q, k, v, ks, vs, wide, lens))


def test_bf16_output_is_the_rounded_fp32_output():
    c = ref.Case([200, 1000], **GQA, seed=2)
    d = device(c)
    a, _ = decoder(c, force_ctas=7, out_dtype=mfa.MFA_OUT_FP32)(*d)
    b, _ = decoder(c, force_ctas=7)(*d)
    assert torch.equal(a.bfloat16(), b)


def test_nothing_past_the_outputs_is_written_and_lse_may_be_left_out():
    c = ref.Case([130, 0, 5], **FIVE, tokens=2, seed=2)
    d, dec = device(c), decoder(c, force_ctas=3)
    want, want_lse = dec(*d)
    n = want.numel()
    buf = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device=DEV)
    lbuf = torch.full((want_lse.numel() + 64,), 7.0, device=DEV)
    dec(*d, out=buf[:n].view(want.shape), lse=lbuf[:want_lse.numel()].view(want_lse.shape))
    assert torch.equal(buf[:n].view(want.shape), want) and bool((buf[n:] == 7).all())
    assert torch.equal(lbuf[:want_lse.numel()].view(want_lse.shape), want_lse) and bool((lbuf[want_lse.numel():] == 7).all())
    out = torch.empty_like(want)
    mfa.mfa_block_decode_run(dec.plan, dec.problem, c.scale_tokens, *d, out, None, dec.workspace)
    assert torch.equal(out, want)


def test_a_plan_from_a_bound_runs_any_lengths():
    c = ref.Case([0, 400, 77, 1], **GQA, columns=16, seed=9)
    d = device(c)
    dec = decoder(c, lens=None, flags=mfa.MFA_PLAN_CHECK)
    check(c, *dec(*d))
    c.seq_lens = torch.tensor([399, 0, 1, 0], dtype=torch.int32)
    c.block_table[0], c.block_table[1] = c.block_table[1].clone(), c.block_table[0].clone()
    d[5], d[6] = c.block_table.to(DEV), c.seq_lens.to(DEV)
    check(c, *dec(*d))


def test_not_finite_queries_stay_in_their_rows():
    c = ref.Case([300, 129], **MFA, seed=10)
    want = ref.decode(c)
    q = c.q.clone()
    q[0, 5, 7], q[0, 40, 0], q[1, 63, 255] = float("nan"), float("inf"), float("-inf")
    d = device(c)
    d[0] = q.to(DEV)
    out, lse = decoder(c, force_ctas=3, flags=mfa.MFA_PLAN_CHECK)(*d)
    for x, h in ((0, 5), (0, 40), (1, 63)):
        out[x, h], lse[x, h] = want[0][x, h].to(DEV).bfloat16(), want[1][x, h].to(DEV)
    check(c, out, lse, want)


def test_a_sequence_with_nan_codes_leaves_the_others_alone():
    """NaN codes among one sequence's tokens reach its own outputs only, whatever shares its CTA."""
    c = ref.Case([300, 64, 200], **MFA, seed=11)
    want = ref.decode(c)
    c.k_cache[c.block_table[1, 0].long(), 0, 3] = 0x7F
    c.v_cache[c.block_table[1, 0].long(), 0, 9] = 0x7F
    for ctas in (1, 2):
        out, lse = decoder(c, force_ctas=ctas)(*device(c))
        assert bool(torch.isnan(out[1].float()).any())
        out[1], lse[1] = want[0][1].to(DEV).bfloat16(), want[1][1].to(DEV)
        check(c, out, lse, want)


def test_bad_pages_read_as_zeros_and_bad_lengths_are_clamped():
    c = ref.Case([200, 130], **GQA, columns=4, seed=12, poison=False)
    dec = decoder(c, lens=None)
    d = device(c)
    for bad in (-1, c.pages, 2 ** 31 - 1):
        table = d[5].clone()
        table[0, 1] = bad
        out, lse = dec(*d[:5], table, d[6])
        assert mfa.mfa_read_device_status(dec.workspace) == mfa.MFA_DEV_BAD_BLOCK
        z = ref.Case([200, 130], **GQA, columns=4, seed=12, poison=False)
        page = z.block_table[0, 1].long()
        z.k_cache[page], z.v_cache[page] = 0, 0
        check(z, out, lse)
    lens = torch.tensor([257, -5], dtype=torch.int32, device=DEV)
    out, lse = dec(*d[:6], lens)
    assert mfa.mfa_read_device_status(dec.workspace) == mfa.MFA_DEV_BAD_LENGTH
    c.seq_lens = torch.tensor([256, 0], dtype=torch.int32)
    check(c, out, lse)


def test_lengths_past_the_plan_are_refused_by_the_device():
    """Planned for 3 short sequences on one CTA, run with lengths that need room for more units."""
    n = 600
    c = ref.Case([0] * (n - 3) + [3] * 3, heads=8, kv_heads=1, dim=128, columns=1, seed=1, poison=False)
    dec = decoder(c, force_ctas=1)
    d = device(c)
    check(c, *dec(*d))
    assert mfa.mfa_read_device_status(dec.workspace) == 0
    dec(*d[:6], torch.full((n,), 5, dtype=torch.int32, device=DEV))
    assert mfa.mfa_read_device_status(dec.workspace) == mfa.MFA_DEV_SCHEDULE


def test_decode_repeats_bit_for_bit_on_any_stream_and_in_a_graph():
    c = ref.Case([700, 64, 1500], **GQA, tokens=2, seed=13)
    d, dec = device(c), decoder(c, lens=None)
    want, want_lse = dec(*d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    dec(*d, out=out, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec(*d, out=out, lse=lse)
    for lens in ([700, 64, 1500], [1, 0, 200]):
        d[6].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(9)
        graph.replay()
        again, again_lse = dec(*d)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_outputs_of_a_call_on_another_stream_stay_until_it_is_done():
    c = ref.Case([500], **GQA, seed=3)
    d, dec, side = device(c), decoder(c), torch.cuda.Stream()
    dec(*d, stream=side)   # (loads what is loaded at a first call)
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        out, lse = dec(*d, stream=stream)
        used, like = {out.data_ptr(), lse.data_ptr()}, (torch.empty(0, dtype=out.dtype), out.shape, lse.shape)
        del out, lse
        new = [torch.empty(like[1], dtype=like[0].dtype, device=DEV), torch.empty(like[2], device=DEV)]
        assert not used & {x.data_ptr() for x in new} or side.query()   # (its memory is free once it is done)
    torch.cuda.synchronize()
    check(c, *dec(*d))


def test_the_first_call_may_be_on_another_stream():
    """The workspace is ready when the decoder is."""
    c = ref.Case([3000, 40], **MFA, seed=4)
    d, side = device(c), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)   # what the current stream still has to do when the workspace is made
    dec = decoder(c, out_dtype=mfa.MFA_OUT_FP32)
    out, lse = dec(*d, stream=side)
    torch.cuda.synchronize()
    check(c, out, lse)
    assert mfa.mfa_read_device_status(dec.workspace) == 0


def test_a_nan_among_the_newest_values_stays_in_its_element_and_head():
    c = ref.Case([70, 200], **GQA, tokens=2, seed=5)
    d, dec = device(c), decoder(c, out_dtype=mfa.MFA_OUT_FP32)
    want, want_lse = dec(*d)
    page, slot, head, element = int(c.block_table[0, 1]), 69 % 64, 2, 17
    d[2][page, head, slot, element] = 0x7F
    out, lse = dec(*d)
    torch.cuda.synchronize()
    group = GQA["heads"] // GQA["kv_heads"]
    assert torch.isnan(out[1, head * group:(head + 1) * group, element]).all()
    out[0:2, head * group:(head + 1) * group, element] = 0   # (the token before it may be reached too)
    want[0:2, head * group:(head + 1) * group, element] = 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_decoders_at_once():
    cases = [ref.Case([900, 300, 50], **MFA, seed=20), ref.Case([1100, 7], **TWELVE, seed=21)]
    decs, devs = [decoder(c) for c in cases], [device(c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                outs[i].append(decs[i](*devs[i]))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        want = ref.decode(c)
        for out, lse in outs[i]:
            check(c, out, lse, want)


def test_the_decoder_checks_its_tensors():
    c = ref.Case([20], **GQA, seed=1)
    d, dec = device(c), decoder(c)
    for i, bad in ((0, d[0].float()), (0, d[0][:, :32]), (1, d[1][:-1]), (2, d[2].view(torch.int8)), (3, d[3].double()),
                   (4, d[4].transpose(0, 1)), (5, d[5][:, :-1]), (6, d[6].long()), (6, d[6].cpu())):
        args = list(d)
        args[i] = bad
        with pytest.raises(ValueError):
            dec(*args)
    with pytest.raises(ValueError):
        dec(*d, out=torch.empty((1, 64, 128), device=DEV))


# ---------------------------------------------------------------------------- append

def append_inputs(counts, positions, shape, seed, specials=False):
    gen = torch.Generator().manual_seed(seed)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    n = int(offsets[-1])
    new = []
    for _ in range(2):
        x = torch.randn((n, shape["kv_heads"], shape["dim"]), generator=gen)
        x = x * torch.exp2((torch.rand((n, shape["kv_heads"], 1), generator=gen) * 2 - 1) * 6)
        if specials:
            kinds = torch.randint(0, 7, (n, shape["kv_heads"]), generator=gen)
            for k, v in ((1, 0.0), (2, -0.0), (3, 448.0), (4, 3e38), (5, 1e-40)):
                x[kinds == k] = v
            x[kinds == 6] *= torch.exp2(torch.randint(-100, 100, (int((kinds == 6).sum()), shape["dim"]), generator=gen).float())
            x = x.clamp(-3.3e38, 3.3e38)
        new.append(x.bfloat16())
    return new, offsets, torch.tensor(positions, dtype=torch.int32)


def run_append(c, new, offsets, positions, mode="offsets", max_new=None, stream=None):
    dec = decoder(c, lens=None)
    pools = [x.clone().to(DEV) for x in (c.k_cache, c.v_cache, c.k_scale, c.v_scale)]
    counts = (offsets[1:] - offsets[:-1]).tolist()
    dec.append(new[0].to(DEV), new[1].to(DEV), positions.to(DEV), c.block_table.to(DEV), *pools,
               offsets=offsets.to(DEV) if mode == "offsets" else None, max_new=max(counts + [0]) if max_new is None else max_new,
               stream=stream)
    torch.cuda.synchronize()
    return dec, pools


def check_append(c, new, offsets, positions, pools):
    for name, x, codes, scale in (("k", new[0], pools[0], pools[2]), ("v", new[1], pools[1], pools[3])):
        wc, ws = ref.append(getattr(c, name + "_cache"), getattr(c, name + "_scale"), c.block_table, positions, x,
                            offsets.tolist(), c.scale_tokens, c.columns * 64)
        assert torch.equal(scale.cpu().view(torch.int32), ws.view(torch.int32)), name
        assert torch.equal(codes.cpu(), wc), (name, (codes.cpu() != wc).nonzero()[:5].tolist())


@pytest.mark.parametrize("shape", [MFA, GQA, SINGLE, TWELVE])
@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("counts, positions", [
    ([1] * 9, [0, 1, 15, 16, 31, 63, 64, 100, -1]),            # one row each, one sequence without
    ([2, 3, 4, 0, 1], [15, 62, 61, 5, 190]),                   # a few, across block and page borders
    ([64, 0, 130, 5, 65], [0, 7, 33, 64, 63]),                 # prompts, from inside a block too
])
def test_append(shape, block, counts, positions):
    c = ref.Case([max(0, p) for p in positions], **shape, scale_tokens=block, columns=4, seed=31)
    new, offsets, pos = append_inputs(counts, positions, shape, seed=block, specials=True)
    _, pools = run_append(c, new, offsets, pos)
    check_append(c, new, offsets, pos, pools)


def test_append_of_equal_counts_needs_no_offsets():
    for tokens in (1, 3):
        c = ref.Case([5, 200, 63], **GQA, scale_tokens=16, tokens=tokens, columns=4, seed=1)
        new, offsets, pos = append_inputs([tokens] * 3, [5, 200, 63], GQA, seed=2)
        _, pools = run_append(c, new, offsets, pos, mode="equal")
        check_append(c, new, offsets, pos, pools)


def test_append_grows_a_scale_that_is_no_power_of_two():
    c = ref.Case([20, 40], **MFA, scale_tokens=64, columns=1, seed=5, pow2=False)
    new, offsets, pos = append_inputs([1, 2], [20, 40], MFA, seed=6)
    new = [x * 64 for x in new]
    _, pools = run_append(c, new, offsets, pos)
    check_append(c, new, offsets, pos, pools)
    # and where the scale stays: quotients by it, not by a power of two
    new = [x / 4096 for x in new]
    _, pools = run_append(c, new, offsets, pos)
    check_append(c, new, offsets, pos, pools)


def test_append_of_what_is_not_finite():
    c = ref.Case([5], **SINGLE, scale_tokens=64, columns=1, seed=5)
    new, offsets, pos = append_inputs([3], [5], SINGLE, seed=6)
    new[0][0, 0, 3], new[0][1, 0, 4], new[0][2, 1] = float("inf"), float("-inf"), float("nan")
    _, pools = run_append(c, new, offsets, pos)
    page = c.block_table[0, 0].long()
    got = pools[0].cpu()[page]
    assert int(got[0, 5, 3]) == 0x7E and int(got[0, 6, 4]) == 0xFE and bool(((got[1, 7] & 0x7F) == 0x7F).all())
    clean = [new[0].clone(), new[1]]
    clean[0][0, 0, 3], clean[0][1, 0, 4], clean[0][2, 1] = 0, 0, 0
    wc, ws = ref.append(c.k_cache, c.k_scale, c.block_table, pos, clean[0], offsets.tolist(), 64, 64)
    assert torch.equal(pools[2].cpu().view(torch.int32), ws.view(torch.int32))
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[0, 5, 3] = keep[0, 6, 4] = False
    keep[1, 7] = False
    assert torch.equal(got[keep], wc[page][keep])


def test_append_reports_and_skips_what_it_cannot_place():
    c = ref.Case([10, 20, 30, 100, 60], **GQA, scale_tokens=16, columns=2, seed=7)
    new, offsets, pos = append_inputs([1, 3, 2, 60, 1], [10, 126, 2 ** 31 - 1, 100, 60], GQA, seed=8)
    c.block_table[0, 0] = c.pages
    dec, pools = run_append(c, new, offsets, pos)
    assert mfa.mfa_read_device_status(dec.workspace) == mfa.MFA_DEV_BAD_BLOCK | mfa.MFA_DEV_BAD_LENGTH
    check_append(c, new, offsets, pos, pools)
    # rows past max_new stay out
    c.block_table[0, 0] = -7
    dec, pools = run_append(c, new, offsets, pos, max_new=8)
    cut = torch.tensor([0, 1, 4, 6, 14, 14])
    kept = [torch.cat([x[:14], x[-1:]]) for x in new]
    cut[5] = 15
    assert mfa.mfa_read_device_status(dec.workspace) == mfa.MFA_DEV_BAD_BLOCK | mfa.MFA_DEV_BAD_LENGTH
    check_append(c, kept, cut, pos, pools)
    # offsets that leave the rows: nothing of that sequence is written
    for bad in ([0, 1, 4, 6, 66, 999], [0, 1, -4, 6, 66, 67], [0, 4, 1, 6, 66, 67]):
        dec = decoder(c, lens=None)
        pools = [x.clone().to(DEV) for x in (c.k_cache, c.v_cache, c.k_scale, c.v_scale)]
        dec.append(new[0].to(DEV), new[1].to(DEV), pos.to(DEV), c.block_table.to(DEV), *pools,
                   offsets=torch.tensor(bad, dtype=torch.int32, device=DEV), max_new=60)
        assert mfa.mfa_read_device_status(dec.workspace) & mfa.MFA_DEV_BAD_LENGTH
        ok = [b for b in range(5) if 0 <= bad[b] <= bad[b + 1] <= 67]
        only = pos.clone()
        only[[b for b in range(5) if b not in ok]] = -1
        rows = {b: (bad[b], bad[b + 1]) for b in ok}
        for name, x, codes in (("k", new[0], pools[0]), ("v", new[1], pools[1])):
            wc, wsc = getattr(c, name + "_cache"), getattr(c, name + "_scale")
            for b in ok:
                one = torch.full_like(pos, -1)
                one[b] = pos[b]
                off = [0] * (b + 1) + [min(60, rows[b][1] - rows[b][0])] * (5 - b)
                wc, wsc = ref.append(wc, wsc, c.block_table, one, x[rows[b][0]:rows[b][1]], off, 16, 128)
            assert torch.equal(codes.cpu(), wc)


def test_a_serving_run_turns_appends_and_decodes():
    """A prompt, then single tokens across a page border, then two tokens at once: rotary positions, append and
    decode chained on one stream, each step against the definitions."""
    shape = GQA
    gen = torch.Generator().manual_seed(50)
    c = ref.Case([0, 0, 0], **shape, scale_tokens=32, columns=4, seed=51)
    codes = {n: (getattr(c, n + "_cache"), getattr(c, n + "_scale")) for n in "kv"}
    pools = [x.clone().to(DEV) for x in (c.k_cache, c.v_cache, c.k_scale, c.v_scale)]
    table = c.block_table.to(DEV)
    rope = mfa.Rope(128, (32, 16, 16))
    held = [0, 0, 0]
    side = torch.cuda.Stream()
    for step, counts in enumerate([[60, 1, 125], [1, 1, 1], [1, 1, 1], [1, 1, 1], [1, 1, 1], [2, 2, 2]]):
        n, T = sum(counts), counts[0] if step else 1
        q = torch.randn((3 * T, 64, 128), generator=gen).bfloat16()
        k = torch.randn((n, 4, 128), generator=gen).bfloat16()
        v = torch.randn((n, 4, 128), generator=gen).bfloat16()
        offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
        kpos = torch.cat([torch.arange(held[b], held[b] + counts[b]) for b in range(3)]).to(torch.int32)
        kpos = torch.stack([kpos, kpos // 7, kpos % 7])
        after = [h + m for h, m in zip(held, counts)]
        qpos = torch.cat([torch.arange(after[b] - T, after[b]) for b in range(3)]).to(torch.int32)
        qpos = torch.stack([qpos, qpos // 7, qpos % 7])
        c.tokens, c.seq_lens = T, torch.tensor(after, dtype=torch.int32)
        dec = decoder(c, lens=None)
        args = [x.to(DEV) for x in (q, k, v, offsets, kpos, qpos, torch.tensor(held, dtype=torch.int32), c.seq_lens)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            qr, _ = rope(args[0], None, args[5])
            _, kr = rope(None, args[1], args[4])
            dec.append(kr, args[2], args[6], table, *pools, offsets=args[3], max_new=max(counts))
            out, lse = dec(qr, pools[0], pools[1], pools[2], pools[3], table, args[7])
        torch.cuda.synchronize()
        assert mfa.mfa_read_device_status(dec.workspace) == 0
        want_k = ref.rope(k, kpos, (32, 16, 16), 1e4, "half")
        assert bool(((kr.cpu().double() - want_k).abs() <= want_k.abs() * 2.0 ** -8 + 2.0 ** -18).all())
        for name, x in (("k", kr.cpu()), ("v", v)):
            codes[name] = ref.append(*codes[name], c.block_table, torch.tensor(held), x, offsets.tolist(), 32, 256)
        assert torch.equal(pools[0].cpu(), codes["k"][0]) and torch.equal(pools[1].cpu(), codes["v"][0])
        (c.k_cache, c.k_scale), (c.v_cache, c.v_scale) = codes["k"], codes["v"]
        c.q = qr.cpu()
        check(c, out, lse)
        held = after
