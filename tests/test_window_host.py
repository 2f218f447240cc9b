"""Windowed decode over a block-scaled cache: what the library checks and plans on the host (no GPU)."""
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
    args = dict(batch=4, max_pages_per_seq=64, num_blocks=256, kv_dtype=mfa.MFA_KV_FP8_E4M3)
    args.update(kw)
    return mfa.make_problem(**args)


@pytest.mark.parametrize("tokens, sinks", [(0, 0), (-1, 0), (1, -1), (0, 4), (-2 ** 31, 0), (1, -2 ** 31)])
def test_windows_without_a_meaning_are_refused(lib, tokens, sinks):
    w = mfa.MfaWindow(tokens, sinks)
    with pytest.raises(mfa.MfaError) as e:
        mfa.mfa_window_decode_plan(problem(), 64, w, None, max_seq_len=64, num_sms=8)
    assert e.value.status == mfa.MFA_ERR_INVALID_ARG
    plan = mfa.mfa_window_decode_plan(problem(), 64, mfa.MfaWindow(1, 0), None, max_seq_len=64, num_sms=8)
    st = lib.mfa_window_decode_run(plan, problem(), 64, w, *[P(0x1000)] * 9, P(0x1000), 1 << 30, None)
    assert st == mfa.MFA_ERR_INVALID_ARG


def test_a_missing_window_is_refused(lib):
    plan = mfa.MfaPlan()
    assert lib.mfa_window_decode_plan(problem(), 64, None, None, 64, 8, 0, 0, plan) == mfa.MFA_ERR_INVALID_ARG
    plan = mfa.mfa_window_decode_plan(problem(), 64, mfa.MfaWindow(8, 0), None, max_seq_len=64, num_sms=8)
    assert lib.mfa_window_decode_run(plan, problem(), 64, None, *[P(0x1000)] * 10, 1 << 30, None) == mfa.MFA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw, block, code", [
    (dict(kv_dtype=mfa.MFA_KV_BF16), 64, mfa.MFA_ERR_UNSUPPORTED), (dict(head_dim=64), 64, mfa.MFA_ERR_UNSUPPORTED),
    (dict(), 48, mfa.MFA_ERR_UNSUPPORTED), (dict(tokens_per_seq=5), 64, mfa.MFA_ERR_INVALID_ARG),
    (dict(num_q_heads=128), 64, mfa.MFA_ERR_UNSUPPORTED), (dict(batch=-1), 64, mfa.MFA_ERR_INVALID_ARG)])
def test_problems_outside_the_cache_are_refused(lib, kw, block, code):
    with pytest.raises(mfa.MfaError) as e:
        mfa.mfa_window_decode_plan(problem(**kw), block, mfa.MfaWindow(64, 0), None, max_seq_len=64, num_sms=8)
    assert e.value.status == code


def test_plans_are_for_one_kind_of_call(lib):
    w = mfa.MfaWindow(100, 4)
    whole = mfa.mfa_block_decode_plan(problem(), 64, [4096] * 4, num_sms=8)
    cut = mfa.mfa_window_decode_plan(problem(), 64, w, [4096] * 4, num_sms=8)
    assert cut.flags & mfa.MFA_PLAN_WINDOW and not whole.flags & mfa.MFA_PLAN_WINDOW
    args = [P(0x1000 * (i + 1)) for i in range(9)]
    assert lib.mfa_block_decode_run(cut, problem(), 64, *args, P(0x10000), 1 << 40, None) == mfa.MFA_ERR_INVALID_ARG
    assert lib.mfa_window_decode_run(whole, problem(), 64, w, *args, P(0x10000), 1 << 40, None) == mfa.MFA_ERR_INVALID_ARG
    with pytest.raises(mfa.MfaError):   # the flag is the plan's, not the caller's
        mfa.mfa_window_decode_plan(problem(), 64, w, [4096] * 4, num_sms=8, flags=mfa.MFA_PLAN_WINDOW)


def test_bad_pointers_are_refused(lib):
    w = mfa.MfaWindow(100, 4)
    plan = mfa.mfa_window_decode_plan(problem(), 64, w, [4096] * 4, num_sms=8)
    good = [0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000, 0x8000, 0x9000, 0x10000]
    for i in range(10):
        for bad in ([None] if i != 8 else []) + [0x1001]:
            args = [P(x) for x in good]
            args[i] = P(bad)
            assert lib.mfa_window_decode_run(plan, problem(), 64, w, *args, 1 << 40, None) == mfa.MFA_ERR_INVALID_ARG
    assert lib.mfa_window_decode_run(plan, problem(), 64, w, *[P(x) for x in good], 64, None) == mfa.MFA_ERR_WORKSPACE


@pytest.mark.parametrize("tokens", [1, 3])
def test_a_plan_counts_the_pages_that_are_seen(lib, tokens):
    """Tiles of two pages: those that hold a token which a new token sees."""
    for window, sinks in ((1, 0), (1, 1), (64, 0), (65, 3), (300, 64), (300, 65), (2 ** 31 - 1, 2 ** 31 - 1), (5, 500), (4000, 2 ** 31 - 1)):
        for L in (1, 2, 63, 64, 65, 130, 400, 601, 1000, 4096):
            see = seen.window_seen(L, tokens, window, sinks).any(0)
            if L < tokens:
                see[:] = True
            last = (L - 1) // 64
            want = sorted({int(t) // 64 for t in see.nonzero()} | {last})
            # the pages up to the sinks' end are kept as they are
            want = sorted(set(want) | {j for j in range(min(-(-sinks // 64), last + 1))})
            plan = mfa.mfa_window_decode_plan(problem(batch=1, tokens_per_seq=tokens, num_q_heads=8, head_dim=128), 64,
                                              mfa.MfaWindow(window, sinks), [L], num_sms=8)
            assert plan.total_tiles == -(-len(want) // 2), (window, sinks, L)


def test_a_plan_from_a_bound_has_room_for_every_length(lib):
    for window, sinks in ((1, 0), (130, 4), (1000, 70)):
        w = mfa.MfaWindow(window, sinks)
        bound = mfa.mfa_window_decode_plan(problem(batch=1), 64, w, None, max_seq_len=4096, num_sms=152)
        for L in range(1, 4097, 37):
            assert mfa.mfa_window_decode_plan(problem(batch=1), 64, w, [L], num_sms=152).total_tiles <= bound.total_tiles


def test_sinks_without_a_window_are_refused(monkeypatch):
    """(The device is not looked at before.)"""
    monkeypatch.setattr(mfa._OnDevice, "__init__", lambda self, device: setattr(self, "_torch", torch))
    with pytest.raises(ValueError, match="sinks"):
        mfa.BlockDecoder(1, 1, 1, sinks=4)


@pytest.mark.parametrize("window, sinks, taken", [(2 ** 32 + 1, 2 ** 33 + 2, (2 ** 31 - 1, 2 ** 31 - 1)),
                                                  (-2 ** 32 + 5, -2 ** 32 + 1, (-1, -1)), (7, 3, (7, 3))])
def test_windows_past_32_bits_stay_what_they_mean(monkeypatch, window, sinks, taken):
    """As large as the library takes (the whole sequence), or refused by it; not what is left of them in 32 bits."""
    class Stop(Exception):
        pass

    def stop(*args, **kw):
        raise Stop

    monkeypatch.setattr(mfa._OnDevice, "__init__", lambda self, device: setattr(self, "_torch", torch))
    monkeypatch.setattr(mfa, "make_problem", stop)
    dec = mfa.BlockDecoder.__new__(mfa.BlockDecoder)
    with pytest.raises(Stop):
        dec.__init__(1, 1, 1, window=window, sinks=sinks)
    assert (dec.window.tokens, dec.window.sinks) == taken
