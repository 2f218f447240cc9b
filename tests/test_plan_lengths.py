"""Plans run lengths that they were not made for: no CTA of theirs can meet more units than it has room for (no GPU)."""
import pytest

import decode_attention_02_gb300 as mfa
from decode_attention_02_gb300 import build

MOST = 256        # units that a CTA has room for
SMS = 152


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return mfa.load_library()


def problem(**kw):
    args = dict(batch=9, max_pages_per_seq=64, num_blocks=4096, kv_dtype=mfa.MFA_KV_FP8_E4M3)
    args.update(kw)
    return mfa.make_problem(**args)


def plan_of(kind, pr, lens, **kw):
    kw = dict(dict(num_sms=SMS), **kw)
    if kind == "tree":
        return mfa.mfa_tree_decode_plan(pr, 64, lens, **kw)
    if kind == "window":
        return mfa.mfa_window_decode_plan(pr, 64, mfa.MfaWindow(100, 4), lens, **kw)
    return mfa.mfa_block_decode_plan(pr, 64, lens, **kw)


def runs_any_lengths(plan, units):
    """Whole units: each has its CTAs.  Even parts: the CTAs take the slots' items in turn.  By cost: the boundaries' cost
    can be raised until a CTA's range holds at most ceil((units - 1) / CTAs) + 1 units."""
    if plan.flags & mfa.MFA_PLAN_UNIT_CLUSTERS:
        return plan.num_ctas % units == 0
    if plan.flags & mfa.MFA_PLAN_EVEN_SPLIT:
        return plan.num_partials <= MOST * plan.num_ctas
    return units - 1 <= (MOST - 2) * plan.num_ctas


SHAPES = [("tree", dict(batch=9, tokens_per_seq=64), 288), ("tree", dict(batch=40, tokens_per_seq=32), 640),
          ("tree", dict(batch=9, tokens_per_seq=64, num_kv_heads=4, head_dim=128), 288),
          ("window", dict(batch=40, num_q_heads=32, num_kv_heads=8, head_dim=128), 320),
          ("window", dict(batch=300, tokens_per_seq=2), 600), ("plain", dict(batch=40, num_q_heads=32, num_kv_heads=8, head_dim=128), 320),
          ("plain", dict(batch=5000, tokens_per_seq=4, num_q_heads=64, num_kv_heads=8, head_dim=128), 40000)]


@pytest.mark.parametrize("kind, kw, units", SHAPES)
@pytest.mark.parametrize("held", [0, 1, 7])
def test_plans_of_empty_sequences_run_any_lengths(lib, kind, kw, units, held):
    pr = problem(**kw)
    for length in (1, 64, 4096):
        plan = plan_of(kind, pr, [length] * held + [0] * (kw["batch"] - held))
        assert plan.num_partials == units + plan.num_ctas - 1
        assert runs_any_lengths(plan, units), (plan.flags, plan.num_ctas)


@pytest.mark.parametrize("kind, kw, units", SHAPES)
def test_a_plan_of_no_tokens_has_ctas_for_its_units(lib, kind, kw, units):
    pr = problem(**kw)
    for plan in (plan_of(kind, pr, [0] * kw["batch"]), plan_of(kind, pr, None, max_seq_len=0)):
        assert plan.num_ctas >= min(units, SMS) and plan.total_tiles == 0


@pytest.mark.parametrize("kind", ["tree", "window", "plain"])
def test_forced_grids_of_empty_sequences_stay_forced(lib, kind):
    for ctas in (1, 3, 200):
        plan = plan_of(kind, problem(), [0] * 9, force_ctas=ctas)
        assert plan.num_ctas == ctas
