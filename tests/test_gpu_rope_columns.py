"""Rotary positions of q and k in one tensor, as far as they do not share memory, on the GPU."""
import pytest
import torch

import decode_attention_02_gb300 as mfa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rows", [1, 2, 9])
def test_columns_of_one_projection_side_by_side(rows):
    """Neighbouring columns, either first, in place and into each other's place; outputs as columns of one tensor."""
    rope, dim = mfa.Rope(64, (16, 8)), 64
    gen = torch.Generator().manual_seed(rows)
    proj = torch.randn((rows, 8 * dim), generator=gen).to(DEV)
    pos = torch.randint(0, 5000, (2, rows), generator=gen).to(torch.int32).to(DEV)
    for a, b in (((0, 6), (6, 8)), ((2, 8), (0, 2)), ((0, 1), (1, 8))):
        def columns(t):
            return t[:, a[0] * dim:a[1] * dim].view(rows, -1, dim), t[:, b[0] * dim:b[1] * dim].view(rows, -1, dim)

        q, k = columns(proj)
        want = rope(q.contiguous(), k.contiguous(), pos)
        into = torch.zeros_like(proj)
        oq, ok = columns(into)
        rope(q, k, pos, q_out=oq, k_out=ok)
        here = proj.clone()
        hq, hk = columns(here)
        rope(hq, hk, pos, q_out=hq, k_out=hk)
        for got in ((oq, ok), (hq, hk)):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    same = proj[:, :2 * dim].view(rows, 2, dim)   # one input for both is only read
    x, y = rope(same, same, pos)
    assert torch.equal(x, y)
    with pytest.raises(mfa.MfaError):
        rope(same, proj[:, 2 * dim:4 * dim].view(rows, 2, dim), pos, k_out=same)
