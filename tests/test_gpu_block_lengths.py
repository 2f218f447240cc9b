"""Decode over a block-scaled cache with lengths other than those of its plan, on the GPU."""
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa
from test_gpu_block import DEV, FIVE, GQA, MFA, SINGLE, TWELVE, WAYS, check, decoder, device

pytestmark = pytest.mark.gpu


def run(way, planned, lens, shape, kw, ctas=0):
    c = ref.Case(lens, **shape, **kw, scale_tokens=32, seed=len(lens) + max(lens))
    dec = decoder(c, lens=planned, force_ctas=ctas, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)
    assert dec.plan.flags & ~mfa.MFA_PLAN_CHECK == WAYS[way], hex(dec.plan.flags)
    rows, dim = c.q.shape[:2], c.q.shape[2]
    out = torch.full((*rows, dim), float("nan"), device=DEV)
    lse = torch.full(rows, float("nan"), device=DEV)
    check(c, *dec(*device(c), out=out, lse=lse))


@pytest.mark.parametrize("way, planned, grown, shape, kw, ctas", [
    ("even", [512], [513], MFA, dict(), 0),                              # one tile more than the plan's parts
    ("even", [512], [8000], MFA, dict(), 0),
    ("even", [1024] * 4, [1025] * 4, MFA, dict(), 0),
    ("even", [1024] * 4, [1025, 3000, 1024, 1], MFA, dict(), 0),
    ("even", [900, 1, 0, 200], [901, 640, 2000, 700], MFA, dict(tokens=3), 12),   # and one that was empty
    ("even", [1300, 100], [1409, 5000], GQA, dict(), 16),
    ("even", [1300, 100], [9000, 5000], TWELVE, dict(tokens=2), 12),
    ("even", [9000, 100, 0, 3000], [9100, 9100, 9100, 9100], GQA, dict(tokens=2), 0),
    ("even", [200], [1000], MFA, dict(), 2),
    ("even", [5000, 3], [5200, 5200], SINGLE, dict(), 48),
    ("even", [3000] + [0] * 70, [3000] + [300] * 70, FIVE, dict(), 0),
    ("clusters", [1024] * 20, [1025] * 20, MFA, dict(), 0),
    ("clusters", [700, 129], [9000, 4000], GQA, dict(tokens=2), 24),
    ("clusters", [300] * 130, [301] * 129 + [4000], MFA, dict(), 0),
    ("cost", [100, 3000, 700, 0, 1], [3001, 3001, 3001, 3001, 3001], GQA, dict(), 7),
    ("cost", [700] * 200, [769] * 199 + [5000], SINGLE, dict(), 0),
])
def test_lengths_past_the_plan(way, planned, grown, shape, kw, ctas):
    run(way, planned, grown, shape, kw, ctas)


@pytest.mark.parametrize("shape, batch", [(MFA, 1), (MFA, 4), (MFA, 20), (GQA, 1), (GQA, 6)])
def test_a_decode_loop_on_the_plan_of_its_first_step(shape, batch):
    """Lengths that grow by one a step, across page and tile borders, under one plan."""
    first, last = 500, 660
    c = ref.Case([last] * batch, **shape, scale_tokens=64, seed=batch)
    dec = decoder(c, lens=[first] * batch, flags=mfa.MFA_PLAN_CHECK, out_dtype=mfa.MFA_OUT_FP32)
    d = device(c)
    for n in range(first, last + 1, 4):
        c.seq_lens = torch.full((batch,), n, dtype=torch.int32)
        out, lse = dec(*d[:6], c.seq_lens.to(DEV), out=torch.full(c.q.shape, float("nan"), device=DEV))
        check(c, out, lse)


def test_a_checked_decode_reports_what_an_append_could_not_place():
    """The decode clears the status word for its own bits; those of an append before it are not lost."""
    c = ref.Case([64, 20], **GQA, scale_tokens=32, columns=2, seed=3, poison=False)
    dec = decoder(c, lens=None, flags=mfa.MFA_PLAN_CHECK)
    d = device(c)
    new = torch.ones((2, 4, 128), dtype=torch.bfloat16, device=DEV)

    def append(positions, table=None, **kw):
        dec.append(new, new, torch.tensor(positions, dtype=torch.int32, device=DEV), d[5] if table is None else table, *d[1:5],
                   **kw)

    bad = d[5].clone()
    bad[0, 1] = c.pages
    for table, positions, bits in ((bad, [64, 20], mfa.MFA_DEV_BAD_BLOCK), (None, [128, 20], mfa.MFA_DEV_BAD_LENGTH)):
        append(positions, table)
        with pytest.raises(mfa.MfaError) as e:
            dec(*d)
        assert e.value.status == mfa.MFA_ERR_DEVICE_CHECK
        assert mfa.mfa_read_device_status(dec.workspace) == bits
        dec(*d)
        append([63, 20])
        dec(*d)                                              # an append with nothing to report
    # both steps at once, on another stream
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    append([64, 20], bad, stream=side)
    with pytest.raises(mfa.MfaError):
        dec(*d[:6], torch.tensor([129, 20], dtype=torch.int32, device=DEV), stream=side)
    assert mfa.mfa_read_device_status(dec.workspace) == mfa.MFA_DEV_BAD_BLOCK | mfa.MFA_DEV_BAD_LENGTH
    # a word of the caller's own is the caller's to read
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    append([64, 20], bad, device_status=word)
    dec(*d)
    assert int(word) == mfa.MFA_DEV_BAD_BLOCK
