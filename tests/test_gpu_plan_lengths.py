"""Decodes with plans that were made for empty or far shorter sequences, on the GPU."""
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa
import seen_reference as seen
import test_gpu_tree as trees
import test_gpu_window as windows

pytestmark = pytest.mark.gpu
DEV = "cuda"
CHECK = dict(flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)


def empty_results(c):
    """Outputs that nothing has been written to."""
    return dict(out=torch.full(c.q.shape, float("nan"), device=DEV), lse=torch.full(c.q.shape[:2], float("nan"), device=DEV))


@pytest.mark.parametrize("shape", [trees.MFA, trees.GQA])
def test_trees_on_a_plan_of_empty_sequences(shape):
    c = trees.case([64, 65, 130, 0, 200, 64, 100, 129, 3], 64, **shape, scale_tokens=32, seed=5)
    dec = trees.decoder(c, lens=[0] * 9, **CHECK)
    out, lse = dec(*trees.device(c), **empty_results(c))
    seen.check(out, lse, trees.expect(c))


@pytest.mark.parametrize("window", [100, 2 ** 31 - 1])
@pytest.mark.parametrize("shape, batch, tokens", [(windows.FIVE, 40, 1), (windows.SINGLE, 200, 2)])
def test_windows_on_a_plan_of_empty_sequences(shape, batch, tokens, window):
    lens = [(37 * i) % 300 for i in range(batch)]
    c = windows.case(lens, window, 4, **shape, tokens=tokens, scale_tokens=32, seed=6)
    dec = windows.decoder(c, window, 4, lens=[0] * batch, **CHECK)
    out, lse = dec(*windows.device(c), **empty_results(c))
    seen.check(out, lse, windows.expect(c, window, 4))


@pytest.mark.parametrize("shape, batch, tokens", [(windows.FIVE, 40, 1), (windows.SINGLE, 200, 2)])
def test_decodes_on_a_plan_of_empty_sequences(shape, batch, tokens):
    lens = [(37 * i) % 300 for i in range(batch)]
    c = ref.Case(lens, **shape, tokens=tokens, scale_tokens=32, seed=7)
    dec = mfa.BlockDecoder(batch, c.columns, c.pages, num_q_heads=c.heads, num_kv_heads=c.kv_heads, head_dim=c.dim,
                           scale_tokens=32, tokens_per_seq=tokens, host_seq_lens=[0] * batch, **CHECK)
    out, lse = dec(*windows.device(c), **empty_results(c))
    seen.check(out, lse, ref.decode(c))


@pytest.mark.parametrize("kind", ["plain", "window", "tree"])
@pytest.mark.parametrize("where", [0, 200, 399])
def test_one_sequence_grows_far_past_a_plan_of_many(kind, where):
    """400 units on two CTAs, one of them of 600 tiles: at a boundary's usual cost one CTA would meet 260 units.
    (The sequences share their pages.)"""
    batch, long = 400, 600 * 128
    one = dict(heads=1, kv_heads=1, dim=128, scale_tokens=64, seed=8, poison=False)
    c = trees.case([long], 1, **one) if kind == "tree" else ref.Case([long], **one)
    lens = [1] * batch
    lens[where] = long
    c.seq_lens = torch.tensor(lens, dtype=torch.int32)
    c.block_table = c.block_table.expand(batch, -1).contiguous()
    gen = torch.Generator().manual_seed(9)
    c.q = torch.randn((batch, 1, 128), generator=gen).bfloat16()
    shape = dict(num_q_heads=1, num_kv_heads=1, head_dim=128, scale_tokens=64, host_seq_lens=[1] * batch, force_ctas=2, **CHECK)
    args = [x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.block_table, c.seq_lens)]
    if kind == "tree":
        dec = mfa.TreeDecoder(batch, c.columns, c.pages, 1, **shape)
        args.append(torch.ones((batch, 1), dtype=torch.int64, device=DEV))
        want = seen.decode(c, lambda b, L: seen.tree_seen(L, 1, [1]), 1, seen.e4m3_and_e5m2)
    else:
        dec = mfa.BlockDecoder(batch, c.columns, c.pages, **shape, **(dict(window=2 ** 31 - 1) if kind == "window" else {}))
        want = ref.decode(c)
    assert dec.plan.num_ctas == 2 and not dec.plan.flags & (mfa.MFA_PLAN_UNIT_CLUSTERS | mfa.MFA_PLAN_EVEN_SPLIT)
    out, lse = dec(*args, **empty_results(c))
    seen.check(out, lse, want)
