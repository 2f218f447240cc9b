"""Attention of drafted trees: what the library checks and plans on the host (no GPU)."""
import ctypes

import pytest
import torch

import decode_attention_02_gb300 as mfa
import seen_reference as seen
from decode_attention_02_gb300 import build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return mfa.load_library()


def problem(**kw):
    args = dict(batch=4, max_pages_per_seq=64, num_blocks=256, kv_dtype=mfa.MFA_KV_FP8_E4M3, tokens_per_seq=32)
    args.update(kw)
    return mfa.make_problem(**args)


def test_masks_of_the_reference():
    assert seen.tree_seen(5, 3, [0b001, 0b011, 0b100]).tolist() == [
        [True, True, True, False, False], [True, True, True, True, False], [True, True, False, False, True]]
    assert seen.tree_seen(2, 3, [0b111, 0, 0b101]).tolist() == [[True, True], [False, False], [False, True]]


@pytest.mark.parametrize("kw, block, code", [
    (dict(tokens_per_seq=0), 64, mfa.MFA_ERR_INVALID_ARG), (dict(tokens_per_seq=65), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(kv_dtype=mfa.MFA_KV_BF16), 64, mfa.MFA_ERR_UNSUPPORTED), (dict(head_dim=64), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(), 48, mfa.MFA_ERR_UNSUPPORTED), (dict(num_q_heads=128), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(num_q_heads=10, num_kv_heads=4), 64, mfa.MFA_ERR_INVALID_ARG), (dict(batch=-1), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(batch=1 << 25, num_q_heads=64), 64, mfa.MFA_ERR_INVALID_ARG)])
def test_problems_are_refused(lib, kw, block, code):
    with pytest.raises(mfa.MfaError) as e:
        mfa.mfa_tree_decode_plan(problem(**kw), block, None, max_seq_len=64, num_sms=8)
    assert e.value.status == code
    plan = mfa.mfa_tree_decode_plan(problem(), 64, None, max_seq_len=64, num_sms=8)
    assert lib.mfa_tree_decode_run(plan, problem(**kw), block, *[P(0x1000)] * 11, 1 << 40, None) == code


def test_plans_are_for_one_kind_of_call(lib):
    tree = mfa.mfa_tree_decode_plan(problem(tokens_per_seq=4), 64, [4096] * 4, num_sms=8)
    plain = mfa.mfa_block_decode_plan(problem(tokens_per_seq=4), 64, [4096] * 4, num_sms=8)
    assert tree.flags & mfa.MFA_PLAN_TREE and not plain.flags & mfa.MFA_PLAN_TREE
    pr, args = problem(tokens_per_seq=4), [P(0x1000 * (i + 1)) for i in range(7)]
    assert lib.mfa_block_decode_run(tree, pr, 64, *args, P(0x8000), P(0x9000), P(0x10000), 1 << 40, None) == mfa.MFA_ERR_INVALID_ARG
    assert lib.mfa_tree_decode_run(plain, pr, 64, *args, P(0x8000), P(0x9000), P(0xA000), P(0x10000), 1 << 40, None) == mfa.MFA_ERR_INVALID_ARG
    for flags in (mfa.MFA_PLAN_TREE, mfa.MFA_PLAN_NO_COMBINE, mfa.MFA_PLAN_EVEN_SPLIT):
        with pytest.raises(mfa.MfaError):
            mfa.mfa_tree_decode_plan(pr, 64, [4096] * 4, num_sms=8, flags=flags)


def test_bad_pointers_are_refused(lib):
    plan = mfa.mfa_tree_decode_plan(problem(), 64, [4096] * 4, num_sms=8)
    good = [0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, 0x9000, 0xA000, 0x10000]
    for i in range(11):
        for bad in ([None] if i != 9 else []) + [0x1001] + ([0x1004] if i == 7 else []):
            args = [P(x) for x in good]
            args[i] = P(bad)
            assert lib.mfa_tree_decode_run(plan, problem(), 64, *args, 1 << 40, None) == mfa.MFA_ERR_INVALID_ARG, (i, bad)
    assert lib.mfa_tree_decode_run(plan, problem(), 64, *[P(x) for x in good], 64, None) == mfa.MFA_ERR_WORKSPACE
    other = mfa.mfa_tree_decode_plan(problem(batch=3), 64, [4096] * 3, num_sms=8)
    assert lib.mfa_tree_decode_run(other, problem(), 64, *[P(x) for x in good], 1 << 40, None) == mfa.MFA_ERR_INVALID_ARG


@pytest.mark.parametrize("heads, kv_heads, tokens, units", [
    (64, 1, 1, 1), (64, 1, 2, 1), (64, 1, 3, 2), (64, 1, 64, 32), (64, 4, 8, 4), (64, 4, 9, 8), (40, 8, 25, 8), (40, 8, 26, 16),
    (24, 2, 10, 2), (24, 2, 64, 14), (3, 3, 64, 3), (43, 1, 64, 32)])
def test_units_of_at_most_128_rows(lib, heads, kv_heads, tokens, units):
    pr = problem(batch=1, num_q_heads=heads, num_kv_heads=kv_heads, head_dim=128, tokens_per_seq=tokens)
    assert mfa.mfa_tree_decode_plan(pr, 64, [1000], num_sms=8).total_tiles == 8 * units


def test_whole_units_need_no_room_for_parts(lib):
    pr = problem(batch=60, tokens_per_seq=64)
    plan = mfa.mfa_tree_decode_plan(pr, 64, [1000] * 60, num_sms=152)
    assert plan.flags & mfa.MFA_PLAN_UNIT_CLUSTERS and plan.num_ctas == 60 * 32 and plan.workspace_bytes < 1 << 16
    few = problem(batch=2, tokens_per_seq=64)
    assert not mfa.mfa_tree_decode_plan(few, 64, [4000] * 2, num_sms=152).flags & mfa.MFA_PLAN_UNIT_CLUSTERS
