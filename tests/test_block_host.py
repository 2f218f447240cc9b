"""Block-scaled cache and rotary positions: what the library checks on the host (no GPU)."""
import ctypes
import math

import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa
from decode_attention_02_gb300 import build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return mfa.load_library()


def problem(**kw):
    args = dict(batch=4, max_pages_per_seq=8, num_blocks=32, kv_dtype=mfa.MFA_KV_FP8_E4M3)
    args.update(kw)
    return mfa.make_problem(**args)


@pytest.mark.parametrize("kw, block, code", [
    (dict(kv_dtype=mfa.MFA_KV_BF16), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(kv_dtype=mfa.MFA_KV_MXFP4), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(kv_dtype=9), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(kv_shared=True), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(head_dim=64), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(head_dim=512), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(page_size=16), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(), 8, mfa.MFA_ERR_UNSUPPORTED),
    (dict(), 48, mfa.MFA_ERR_UNSUPPORTED),
    (dict(), 128, mfa.MFA_ERR_UNSUPPORTED),
    (dict(), 0, mfa.MFA_ERR_INVALID_ARG),
    (dict(num_q_heads=128), 64, mfa.MFA_ERR_UNSUPPORTED),          # 128 query heads a key head
    (dict(num_q_heads=65537, num_kv_heads=65537, head_dim=128), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(num_q_heads=10, num_kv_heads=4), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(num_q_heads=0), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(tokens_per_seq=0), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(tokens_per_seq=5), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(out_dtype=2), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(softmax_scale=0.0), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(softmax_scale=float("nan")), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(softmax_scale=float("inf")), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(batch=-1), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(max_pages_per_seq=1 << 25), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(num_blocks=1 << 29, num_kv_heads=4), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(batch=1 << 28), 64, mfa.MFA_ERR_INVALID_ARG),
])
def test_problems_outside_the_cache_are_refused(lib, kw, block, code):
    pr = problem(**kw)
    with pytest.raises(mfa.MfaError) as e:
        mfa.mfa_block_decode_plan(pr, block, None, max_seq_len=64, num_sms=8)
    assert e.value.status == code
    st = lib.mfa_block_kv_append(pr, block, *[P(0x1000)] * 2, 4, None, 0, *[P(0x1000)] * 6, None, None)
    assert st == code


@pytest.mark.parametrize("kw, rows, units", [
    (dict(), 64, 4),                                                       # 64 heads over one
    (dict(tokens_per_seq=3), 64, 12),                                      # each token a unit of its own
    (dict(num_kv_heads=4, head_dim=128, tokens_per_seq=4), 64, 16),        # 16 heads x 4 tokens in a unit
    (dict(num_q_heads=40, num_kv_heads=8, head_dim=128), 8, 32),           # 5 rows, padded to 8
    (dict(num_q_heads=24, num_kv_heads=1, tokens_per_seq=3), 48, 8),       # 2 + 1 tokens
])
def test_plan_sizes(lib, kw, rows, units):
    pr = problem(**kw)
    plan = mfa.mfa_block_decode_plan(pr, 32, [0, 1, 128, 512], num_sms=152)
    assert plan.total_tiles == 6 * units // 4
    # a tile a CTA, or the longest sequence's four tiles on the four CTAs of a cluster
    ctas = {mfa.MFA_PLAN_EVEN_SPLIT: plan.total_tiles, mfa.MFA_PLAN_UNIT_CLUSTERS: 4 * units}
    assert plan.num_ctas == ctas[plan.flags]
    assert plan.num_partials == units + plan.num_ctas - 1
    o_end = (256 + plan.num_partials * rows * pr.head_dim * 4 + 255) // 256 * 256
    lse_end = (o_end + plan.num_partials * rows * 4 + 255) // 256 * 256
    assert plan.workspace_bytes == (lse_end + units * 8 + 255) // 256 * 256


def test_plan_grids(lib):
    big = problem(batch=4000, max_pages_per_seq=64, num_blocks=4000 * 64)
    plan = mfa.mfa_block_decode_plan(big, 64, [1] * 4000, num_sms=8)
    assert plan.num_ctas > 8                                  # no CTA meets more units than it has room for
    assert 4000 / plan.num_ctas < 255
    with pytest.raises(mfa.MfaError):
        mfa.mfa_block_decode_plan(big, 64, [1] * 4000, num_sms=8, force_ctas=8)
    assert mfa.mfa_block_decode_plan(problem(), 64, [0] * 4, num_sms=152).num_ctas == 1
    assert mfa.mfa_block_decode_plan(problem(batch=0), 64, [], num_sms=152).num_ctas == 1
    for bad in ([1, 2, 3, 513], [1, 2, 3, -1]):
        with pytest.raises(mfa.MfaError):
            mfa.mfa_block_decode_plan(problem(), 64, bad, num_sms=8)
    with pytest.raises(ValueError):
        mfa.mfa_block_decode_plan(problem(), 64, [1, 2, 3], num_sms=8)
    with pytest.raises(mfa.MfaError):
        mfa.mfa_block_decode_plan(problem(), 64, None, max_seq_len=513, num_sms=8)
    with pytest.raises(mfa.MfaError):
        mfa.mfa_block_decode_plan(problem(), 64, None, max_seq_len=64, num_sms=8, flags=mfa.MFA_PLAN_NO_COMBINE)


def test_run_refuses_before_touching_the_device(lib):
    pr = problem()
    plan = mfa.mfa_block_decode_plan(pr, 64, [10, 20, 30, 40], num_sms=8)
    # q, k, v, k_scale, v_scale, table, lens, out, lse, workspace
    good = [0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, 0x9000, 0x10000]

    def call(ptrs=good, pl=plan, p=pr, block=64, ws=plan.workspace_bytes):
        return lib.mfa_block_decode_run(pl, p, block, *[P(x) if x else None for x in ptrs], ctypes.c_uint64(ws), None)

    for i, off in ((0, 8), (1, 8), (2, 8), (3, 8), (4, 8), (5, 2), (6, 2), (7, 8), (8, 2), (9, 128)):
        bad = list(good)
        bad[i] += off
        assert call(bad) == mfa.MFA_ERR_INVALID_ARG, i
        if i != 8:                                            # lse may be left out
            bad[i] = None
            assert call(bad) == mfa.MFA_ERR_INVALID_ARG, i
    assert call(ws=plan.workspace_bytes - 1) == mfa.MFA_ERR_WORKSPACE
    assert call(p=problem(batch=5)) == mfa.MFA_ERR_INVALID_ARG
    assert call(p=problem(head_dim=128)) == mfa.MFA_ERR_INVALID_ARG          # a plan for another width
    assert call(block=24) == mfa.MFA_ERR_UNSUPPORTED
    assert lib.mfa_block_decode_run(None, pr, 64, *[P(x) for x in good], ctypes.c_uint64(plan.workspace_bytes),
                                    None) == mfa.MFA_ERR_INVALID_ARG
    empty = problem(batch=0)
    assert call([None] * 10, mfa.mfa_block_decode_plan(empty, 64, [], num_sms=8), empty, ws=0) == mfa.MFA_OK


def test_append_refuses_before_touching_the_device(lib):
    pr = problem()
    good = [0x1000, 0x2000, 4, 0x3000, 1, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, 0x9000, 0xA000]
    # k_new, v_new, num_new, offsets, max_new, positions, table, k, v, k_scale, v_scale, status

    def call(a=good, p=pr):
        a = [x if i in (2, 4) else (P(x) if x else None) for i, x in enumerate(a)]
        return lib.mfa_block_kv_append(p, 64, *a, None)

    for i, off in ((0, 8), (1, 8), (3, 2), (5, 2), (6, 2), (7, 8), (8, 8), (9, 8), (10, 8), (11, 2)):
        bad = list(good)
        bad[i] += off
        assert call(bad) == mfa.MFA_ERR_INVALID_ARG, i
        if i not in (3, 11):
            bad[i] = None
            assert call(bad) == mfa.MFA_ERR_INVALID_ARG, i
    for i, v in ((2, -1), (4, 0), (4, -3)):
        bad = list(good)
        bad[i] = v
        assert call(bad) == mfa.MFA_ERR_INVALID_ARG, (i, v)
    bad = list(good)
    bad[3] = None                                             # T rows each: 4 rows for 4 sequences, not 5
    bad[2] = 5
    assert call(bad) == mfa.MFA_ERR_INVALID_ARG
    bad[2] = 0
    bad[3] = 0x3000
    assert call(bad) == mfa.MFA_OK                            # no rows: nothing enqueued
    assert call([None, None, 0, None, 0] + [None] * 7, problem(batch=0)) == mfa.MFA_OK


# ---------------------------------------------------------------------------- rotary positions

def config(head_dim=128, sections=(32, 16, 16), pairing=0, flags=0, theta=1e4, scale=1.0, axes=None, rotary=None):
    full = (list(sections) + [0] * 4)[:4]
    return mfa.MfaRopeConfig(head_dim, 2 * sum(sections) if rotary is None else rotary,
                             len(sections) if axes is None else axes, (ctypes.c_int32 * 4)(*full), pairing, flags,
                             theta, scale)


@pytest.mark.parametrize("kw, code", [
    (dict(head_dim=100), mfa.MFA_ERR_INVALID_ARG),             # more pairs than the head holds
    (dict(head_dim=1024), mfa.MFA_ERR_UNSUPPORTED),
    (dict(sections=(0, 0)), mfa.MFA_ERR_INVALID_ARG),
    (dict(sections=(70, -6)), mfa.MFA_ERR_INVALID_ARG),
    (dict(rotary=126), mfa.MFA_ERR_INVALID_ARG),
    (dict(sections=(2,), rotary=5), mfa.MFA_ERR_INVALID_ARG),
    (dict(axes=0), mfa.MFA_ERR_INVALID_ARG),
    (dict(axes=5), mfa.MFA_ERR_INVALID_ARG),
    (dict(axes=2), mfa.MFA_ERR_INVALID_ARG),                   # pairs on an axis past num_axes
    (dict(pairing=2), mfa.MFA_ERR_INVALID_ARG),
    (dict(flags=8), mfa.MFA_ERR_INVALID_ARG),
    (dict(theta=0.5), mfa.MFA_ERR_INVALID_ARG),
    (dict(theta=float("nan")), mfa.MFA_ERR_INVALID_ARG),
    (dict(theta=float("inf")), mfa.MFA_ERR_INVALID_ARG),
    (dict(scale=0.0), mfa.MFA_ERR_INVALID_ARG),
    (dict(scale=17.0), mfa.MFA_ERR_INVALID_ARG),
])
def test_rope_configs_that_mean_nothing_are_refused(lib, kw, code):
    c = config(**kw)
    with pytest.raises(mfa.MfaError) as e:
        mfa.mfa_rope_table(c)
    assert e.value.status == code
    assert lib.mfa_rope_run(c, P(0x1000), P(0x1000), 1, 0, 0, None, None, None) == code


@pytest.mark.parametrize("sections, flags", [((64,), 0), ((32, 16, 16), 0), ((24, 20, 20), mfa.MFA_ROPE_INTERLEAVED),
                                             ((8, 0, 3, 5), mfa.MFA_ROPE_INTERLEAVED | mfa.MFA_ROPE_OWN_SPECTRUM),
                                             ((1, 30), mfa.MFA_ROPE_OWN_SPECTRUM)])
def test_rope_table_holds_the_frequencies(lib, sections, flags):
    for theta, scale in ((1e4, 1.0), (5e6, 0.25), (1.0, 16.0)):
        t = mfa.mfa_rope_table(config(sections=sections, flags=flags, theta=theta, scale=scale))
        axes = ref.rope_axes(sections, bool(flags & mfa.MFA_ROPE_INTERLEAVED))
        assert [x.axis for x in t] == axes and all(x.reserved == 0 for x in t)
        seen = [0] * len(sections)
        for i, (x, a) in enumerate(zip(t, axes)):
            power = seen[a] / sections[a] if flags & mfa.MFA_ROPE_OWN_SPECTRUM else i / sum(sections)
            seen[a] += 1
            turns = math.pow(theta, -power) * scale / (2 * math.pi)
            # doubles: pow, two products and 2^64 times the part, each half a step of turns <= 2.6
            assert abs(x.turns / 2.0 ** 64 - turns % 1.0) <= 4 * 2.0 ** -52 * max(1.0, turns), i


def test_rope_run_refuses_before_touching_the_device(lib):
    c = config()

    def rows(i=0x10000, o=0x900000, si=512, so=512, heads=4):
        return mfa.MfaRopeRows(i, o, si, so, heads)

    def call(q, k=None, table=0x1000, pos=0x2000, n=8, dtype=0, inv=0):
        return lib.mfa_rope_run(c, P(table) if table else None, P(pos) if pos else None, n, dtype, inv, q, k, None)

    bad = [rows(i=None), rows(o=None), rows(i=0x10001), rows(o=0x900001), rows(si=511), rows(so=500), rows(heads=-1),
           rows(o=0x10000, so=520),                   # in place with another stride
           rows(o=0x10010),                           # shifted onto itself
           rows(o=0x10000 + 512 * 2 * 3 + 2),         # three rows and one element on
           rows(si=1 << 50)]
    for r in bad:
        assert call(r) == mfa.MFA_ERR_INVALID_ARG
        assert call(None, r) == mfa.MFA_ERR_INVALID_ARG
    ok = rows()
    assert call(ok, table=None) == mfa.MFA_ERR_INVALID_ARG
    assert call(ok, table=0x1008) == mfa.MFA_ERR_INVALID_ARG
    assert call(ok, pos=None) == mfa.MFA_ERR_INVALID_ARG
    assert call(ok, pos=0x2002) == mfa.MFA_ERR_INVALID_ARG
    assert call(ok, n=-1) == mfa.MFA_ERR_INVALID_ARG
    assert call(ok, dtype=2) == mfa.MFA_ERR_INVALID_ARG
    assert call(ok, inv=2) == mfa.MFA_ERR_INVALID_ARG
    assert call(rows(i=0x10002), dtype=1) == mfa.MFA_ERR_INVALID_ARG       # fp32 rows at a 2-byte address
    # nothing to do: nothing enqueued
    assert call(None) == mfa.MFA_OK
    assert call(rows(heads=0)) == mfa.MFA_OK
    assert call(ok, n=0) == mfa.MFA_OK


def test_reference_rope_keeps_lengths_and_relative_angles():
    """The oracle itself: turning keeps each pair's norm, and dot products depend on the distance."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((2, 1, 8), generator=g).double()
    pos = torch.tensor([[5, 9]], dtype=torch.int32)
    y = ref.rope(x, pos, (4,), 1e4, "half")
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), atol=1e-12)
    z = ref.rope(x, pos + 100, (4,), 1e4, "half")
    assert torch.allclose((y[0] * y[1]).sum(), (z[0] * z[1]).sum(), atol=1e-12)
    assert torch.allclose(ref.rope(y, pos, (4,), 1e4, "half", sign=-1), x, atol=1e-12)


def test_reference_append_and_decode_by_hand():
    """The oracle itself, on a block that is filled in two goes and read back."""
    cache = torch.full((1, 1, 64, 128), 0x7F, dtype=torch.uint8)
    scale = torch.full((1, 1, 4), float("nan"))
    table = torch.zeros((1, 1), dtype=torch.int32)
    one = torch.full((1, 1, 128), 448.0).bfloat16()
    c, s = ref.append(cache, scale, table, torch.tensor([16]), one, [0, 1], 16, 64)
    assert float(s[0, 0, 1]) == 1.0 and int(c[0, 0, 16, 0]) == 0x7E and bool(torch.isnan(s[0, 0, 0]))
    c, s = ref.append(c, s, table, torch.tensor([17]), one * 4, [0, 1], 16, 64)
    assert float(s[0, 0, 1]) == 4.0                                        # the scale rose
    assert float(c[0, 0, 16, 0].view(torch.float8_e4m3fn)) * 4.0 == 448.0  # and the older row kept its value
    assert float(c[0, 0, 17, 0].view(torch.float8_e4m3fn)) * 4.0 == 1792.0
    assert int(c[0, 0, 18, 0]) == 0x7F
    case = ref.Case([1], kv_heads=1, heads=2, dim=128, scale_tokens=16)
    out, lse, _, _ = ref.decode(case)
    v, _ = case.rows("v", 0, 1)
    assert torch.equal(out[0, 0], v[0, 0])
