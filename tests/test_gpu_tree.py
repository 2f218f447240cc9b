"""Attention of drafted trees over a block-scaled cache on the GPU, against its definition in 64 bits."""
import random

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


def draft(T, rng):
    """Masks of a random tree: node i hangs from one of the nodes before it, or from the last token of the cache."""
    masks = []
    for i in range(T):
        parent = rng.randint(-1, i - 1)
        masks.append((masks[parent] if parent >= 0 else 0) | 1 << i)
    return masks


def case(lens, T, masks="trees", **kw):
    c = ref.Case(lens, tokens=T, **kw)
    rng = random.Random(T + len(lens))
    if masks == "trees":
        c.masks = [draft(T, rng) for _ in lens]
    elif masks == "any":      # any bits, ones past T among them, and nodes that see no node
        c.masks = [[rng.choice([0, rng.getrandbits(64)]) for _ in range(T)] for _ in lens]
    else:
        c.masks = [list(masks) for _ in lens]
    c.tree = torch.tensor([[m - (1 << 64) if m >> 63 else m for m in r] for r in c.masks], dtype=torch.int64).reshape(len(lens), T)
    return c


def decoder(c, lens="plan", **kw):
    host = c.seq_lens.tolist() if lens == "plan" else lens
    return mfa.TreeDecoder(len(c.seq_lens), c.columns, c.pages, c.tokens, num_q_heads=c.heads, num_kv_heads=c.kv_heads,
                           head_dim=c.dim, scale_tokens=c.scale_tokens, host_seq_lens=host, **kw)


def device(c):
    return [x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.block_table, c.seq_lens, c.tree)]


def expect(c, **kw):
    return seen.decode(c, lambda b, L: seen.tree_seen(L, c.tokens, c.masks[b]), c.tokens, seen.e4m3_and_e5m2, **kw)


CHECK = dict(flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)


@pytest.mark.parametrize("shape, block", [(MFA, 64), (MFA, 16), (GQA, 32), (GQA, 64), (FIVE, 16), (TWELVE, 32), (SINGLE, 64)])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 31])
def test_trees(shape, block, T):
    """Lengths around pages and tiles, trees over their borders, sequences shorter than their tree, empty ones."""
    c = case([T, T + 1, 64, 65, 0, 127, 128, 129, 130, 1, 191, 192, 128 + T, 517], T, **shape, scale_tokens=block, seed=T)
    out, lse = decoder(c, **CHECK)(*device(c))
    seen.check(out, lse, expect(c))


@pytest.mark.parametrize("shape", [MFA, GQA, TWELVE])
@pytest.mark.parametrize("T", [63, 64])
def test_the_largest_trees(shape, T):
    c = case([T, 64, 200, 300, 40, 1025], T, **shape, seed=T)
    out, lse = decoder(c, flags=mfa.MFA_PLAN_CHECK)(*device(c))
    seen.check(out, lse, expect(c))


@pytest.mark.parametrize("T", [1, 5, 64])
@pytest.mark.parametrize("shape", [MFA, FIVE])
def test_any_masks(shape, T):
    """Bits past the tree, nodes that see no node or not themselves; rows that see nothing where the tree is all there is."""
    c = case([T, 70, 130, 1, 64, 257], T, masks="any", **shape, scale_tokens=32, seed=T)
    out, lse = decoder(c, **CHECK)(*device(c))
    seen.check(out, lse, expect(c))


def test_a_chain_is_the_decode_of_several_new_tokens():
    c = case([5, 700, 1300, 64, 2], 4, masks=[1, 3, 7, 15], **GQA, scale_tokens=16, seed=4)
    d = device(c)
    dec = mfa.BlockDecoder(5, c.columns, c.pages, num_q_heads=64, num_kv_heads=4, head_dim=128, scale_tokens=16, tokens_per_seq=4,
                           host_seq_lens=c.seq_lens.tolist(), out_dtype=mfa.MFA_OUT_FP32)
    want, want_lse = ref.decode(c)[:2]
    for out, lse in (dec(*d[:7]), decoder(c, **CHECK)(*d)):
        seen.check(out, lse, expect(c))
        assert torch.allclose(lse.cpu().double(), want_lse, atol=1e-4)


@pytest.mark.parametrize("ctas", [1, 2, 5, 17, 64])
@pytest.mark.parametrize("shape, T", [(MFA, 3), (GQA, 20), (TWELVE, 11)])
def test_split_over_any_grid(shape, T, ctas):
    c = case([700, 0, 129, 1, 1300], T, **shape, scale_tokens=32, seed=ctas)
    out, lse = decoder(c, force_ctas=ctas, **CHECK)(*device(c))
    seen.check(out, lse, expect(c))


@pytest.mark.parametrize("kw", [dict(spread=12.0), dict(spread=6.0, pow2=False), dict(q_spread=10.0), dict(pow2=False)])
@pytest.mark.parametrize("shape", [MFA, GQA])
def test_scales_and_heads_far_apart(shape, kw):
    c = case([333, 1024], 9, **shape, scale_tokens=16, seed=3, **kw)
    c.k_scale /= 2.0 ** kw.get("spread", 0.0)     # scores of an ordinary size from the largest keys
    c.q = (c.q.float() / 2.0 ** kw.get("q_spread", 0.0)).bfloat16()
    out, lse = decoder(c, force_ctas=3, **CHECK)(*device(c))
    seen.check(out, lse, expect(c))


def test_peaked_and_growing_scores():
    """Scores that climb along the sequence (references rise again and again) and fall behind their peak."""
    c = case([900, 640], 6, **MFA, scale_tokens=16, seed=8)
    c.q = (c.q.float() * 4).bfloat16()
    for b in range(2):
        for t in range(0, int(c.seq_lens[b]), 16):
            page = c.block_table[b, t // 64]
            c.k_scale[page, 0, t % 64 // 16] *= (1.0 + t / 200.0) if b == 0 else (4.0 - t / 200.0)
    out, lse = decoder(c, force_ctas=2, **CHECK)(*device(c))
    seen.check(out, lse, expect(c))


@pytest.mark.parametrize("where", [0, 5, 1000])
@pytest.mark.parametrize("over", [6.0, 12.0, 16.0])
def test_small_weights_behind_a_far_larger_one_keep_theirs(over, where):
    """One token far over 8000 others, its value next to nothing: the others are what the rows come out as."""
    H, d, L = 8, 128, 8064
    c = case([L], 16, heads=H, kv_heads=1, dim=d, seed=5, poison=False, spread=0.0)
    gen = torch.Generator().manual_seed(1)
    c.q = torch.ones_like(c.q)
    k = torch.randn((c.pages, 1, 64, d), generator=gen) / 16
    v = 1 + torch.randn((c.pages, 1, 64, d), generator=gen) / 8
    page, slot = int(c.block_table[0, where // 64]), where % 64
    k[page, 0, slot] += over / d ** 0.5
    v[page, 0, slot] = 2.0 ** -8
    for name, x in (("k", k), ("v", v)):
        s = torch.full((c.pages, 1, 1), 2.0 ** -6)
        setattr(c, name + "_cache", (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).contiguous())
        setattr(c, name + "_scale", s)
    out, lse = decoder(c, **CHECK)(*device(c))
    want = expect(c)
    seen.check(out, lse, want)
    assert float((out.cpu().double() - want[0]).norm() / want[0].norm()) < 2.0 ** -8


@pytest.mark.parametrize("rise", [20, -20, 60])
def test_a_value_scale_far_from_the_others(rise):
    """The last block's scale 2^rise times what it was: the nodes that see none of it keep their precision."""
    c = case([200, 333], 20, **GQA, scale_tokens=32, seed=rise + 100, poison=False)
    for b, L in enumerate(c.seq_lens.tolist()):
        page, block = int(c.block_table[b, (L - 1) // 64]), (L - 1) % 64 // 32
        c.v_scale[page, :, block] *= 2.0 ** rise
    out, lse = decoder(c, **CHECK)(*device(c))
    seen.check(out, lse, expect(c))


def test_blocks_of_zero_values_stay_in_the_sums():
    c = case([512, 700, 128, 40], 5, **MFA, scale_tokens=32, seed=9, poison=False)
    for b, blocks in enumerate(([0, 1, 2, 3, 4, 5, 6], [3, 4, 9, 20], [0, 1, 2, 3], [1])):
        for k in blocks:
            page, at = int(c.block_table[b, k // 2]), k % 2
            c.v_cache[page, :, 32 * at:32 * at + 32] = 0
            c.v_scale[page, :, at] = 2.0 ** -126
    for ctas in (2, 0):
        out, lse = decoder(c, force_ctas=ctas, **CHECK)(*device(c))
        seen.check(out, lse, expect(c))


def test_a_bad_row_and_a_bad_key_spoil_their_own():
    """An infinity or NaN in q: its row.  A NaN key of a node: the rows that see it."""
    c = case([300], 6, masks=[1, 3, 5, 9, 17, 33], **GQA, seed=2)
    d = device(c)
    good, good_lse = decoder(c, **CHECK)(*d)
    q = d[0].clone()
    q[2, 5, 7], q[4, 60, 100] = float("nan"), float("inf")
    out, lse = decoder(c, **CHECK)(q, *d[1:])
    bad = torch.zeros((6, 64), dtype=torch.bool)
    bad[2, 5] = bad[4, 60] = True
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], good_lse[~bad])
    k = d[1].clone()
    page, slot = int(c.block_table[0, 296 // 64]), 296 % 64      # node 2
    k[page, 1, slot, 3] = 0x7F
    out, lse = decoder(c, **CHECK)(d[0], k, *d[2:])
    bad = torch.zeros((6, 64), dtype=torch.bool)
    bad[2, 16:32] = True
    assert bool(out[bad].isnan().all()) and torch.equal(out[~bad], good[~bad])


def test_long_and_many_sequences():
    c = case([70001, 33], 12, heads=8, kv_heads=1, dim=128, seed=4, poison=False)
    seen.check(*decoder(c, flags=mfa.MFA_PLAN_CHECK)(*device(c)), expect(c))
    rng = np.random.default_rng(5)
    c = case(rng.integers(0, 9, 500).tolist(), 5, heads=16, kv_heads=8, dim=128, columns=1, seed=6)
    for kw in (dict(), dict(force_ctas=40)):
        seen.check(*decoder(c, flags=mfa.MFA_PLAN_CHECK, **kw)(*device(c)), expect(c))


def test_lengths_other_than_planned_and_bf16_rounding():
    c = case([700, 129, 2000], 10, **TWELVE, scale_tokens=32, seed=7, poison=False)
    d = device(c)
    dec = decoder(c, lens=[100, 100, 100], **CHECK)
    a, lse = dec(*d)
    seen.check(a, lse, expect(c))
    same = decoder(c, lens=[100, 100, 100])
    assert torch.equal(same(*d)[0], a.bfloat16())
    c.seq_lens = torch.tensor([9, 2000, 64], dtype=torch.int32).clamp(max=700)
    seen.check(*dec(*d[:6], c.seq_lens.to(DEV), d[7]), expect(c))


def test_bad_pages_and_lengths_are_reported():
    c = case([500, 300], 5, **GQA, seed=1, poison=False)
    d, dec = device(c), decoder(c, flags=mfa.MFA_PLAN_CHECK)
    table = d[5].clone()
    table[0, 2] = c.pages
    for args, bit in (((*d[:5], table, *d[6:]), mfa.MFA_DEV_BAD_BLOCK),
                      ((*d[:6], torch.tensor([500, -1], dtype=torch.int32, device=DEV), d[7]), mfa.MFA_DEV_BAD_LENGTH),
                      ((*d[:6], torch.tensor([500, 1 << 20], dtype=torch.int32, device=DEV), d[7]), mfa.MFA_DEV_BAD_LENGTH)):
        with pytest.raises(mfa.MfaError):
            dec(*args)
        assert mfa.mfa_read_device_status(dec.workspace) & bit
    seen.check(*dec(*d), expect(c))


def test_nothing_past_the_outputs_is_written_and_no_state_stays():
    c = case([130, 0, 5, 900], 3, **FIVE, seed=2)
    d, dec, rows = device(c), decoder(c, force_ctas=3), 12
    big, big_lse = torch.full((rows + 4, 40, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((rows + 4, 40), 7.0, device=DEV)
    first = dec(*d)
    dec(*d, out=big[:rows], lse=big_lse[:rows])
    assert torch.equal(big[:rows], first[0]) and torch.equal(big_lse[:rows], first[1])
    assert bool((big[rows:] == 7).all()) and bool((big_lse[rows:] == 7).all())


def test_refusals():
    c = case([130, 70], 3, **GQA, seed=2)
    d, dec = device(c), decoder(c)
    for i, bad in ((7, d[7].int()), (7, d[7][:, :2]), (7, d[7][:1]), (7, d[7].cpu()), (7, d[7].t().contiguous().t()), (0, d[0][:5]),
                   (6, d[6].long()), (1, d[1].float())):
        args = list(d)
        args[i] = bad
        with pytest.raises(ValueError):
            dec(*args)
    with pytest.raises(mfa.MfaError):
        mfa.TreeDecoder(1, 4, 4, 65)
    with pytest.raises(mfa.MfaError):
        mfa.TreeDecoder(1, 4, 4, 0)
    with pytest.raises(ValueError):
        dec.append(torch.zeros((5, 4, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((5, 4, 128), dtype=torch.bfloat16, device=DEV),
                   d[6], *[d[i] for i in (5, 1, 2, 3, 4)])


def test_in_a_graph_and_on_another_stream():
    c = case([900, 2000, 77, 0], 14, **GQA, scale_tokens=32, seed=8)
    d, dec, want = device(c), decoder(c), expect(c)
    first = dec(*d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = dec(*d, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = dec(*d)
    for _ in range(3):
        held[0].zero_()
        graph.replay()
    torch.cuda.synchronize()
    for got in (first, other, held):
        seen.check(*got, want)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("flags", [0, mfa.MFA_PLAN_EARLY_METADATA])
def test_behind_kernels_that_write_its_inputs(flags):
    """Calls that follow one another without a wait: q and the masks of each are written by the kernel before it."""
    c = case([900, 333, 77], 7, **MFA, scale_tokens=64, seed=3)
    d, dec = device(c), decoder(c, flags=flags, force_ctas=20)
    want = dec(*d)
    q, tree = torch.zeros_like(d[0]), torch.zeros_like(d[7])
    outs = []
    for _ in range(5):
        q.zero_()
        tree.zero_()
        q.copy_(d[0])
        tree.copy_(d[7])
        outs.append(dec(q, *d[1:7], tree))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in outs)
