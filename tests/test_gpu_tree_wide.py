"""A drafted tree's rows past 32 bits of bytes within a unit, on the GPU."""
import math

import pytest
import torch

import decode_attention_02_gb300 as mfa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_rows_of_a_unit_further_apart_than_two_gigabytes():
    """64 nodes of 131072 query heads over 65536 of 256: node 63's row lies 4 GB behind node 0's, in one unit.  A sample of heads
    against 64 bits."""
    T, G, d = 64, 65536, 256
    H = 2 * G
    gen = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn((T, H, d), generator=gen, device=DEV, dtype=torch.bfloat16)
    codes = [torch.randint(0, 256, (1, G, 64, d), generator=gen, device=DEV, dtype=torch.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 127) > 0x60] = 0x28   # values of 32 at most: scores of a few units
    scales = [torch.full((1, G, 1), x, device=DEV) for x in (0.125, 1.0)]
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    masks = [(1 << (i + 1)) - 1 for i in range(T)]
    tree = torch.tensor([[m - (1 << 64) if m >> 63 else m for m in masks]], dtype=torch.int64, device=DEV)
    dec = mfa.TreeDecoder(1, 1, 1, T, num_q_heads=H, num_kv_heads=G, head_dim=d, host_seq_lens=[T], flags=mfa.MFA_PLAN_CHECK)
    out, lse = dec(q, *codes, *scales, table, lens, tree)
    torch.cuda.synchronize()
    seen = torch.ones((T, T), dtype=torch.bool, device=DEV).tril()
    for h in (0, 1, 40000, 65535, 65536, 99999, H - 2, H - 1):
        k, v = (c[0, h // 2].view(torch.float8_e4m3fn).double() * float(s[0, h // 2, 0]) for c, s in zip(codes, scales))
        s = (q[:, h].double() @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
        p = torch.softmax(s, -1)
        want, size = p @ v, p @ v.abs()
        # each weight is off by 2^-7 of itself, or 2^-10 of its row's largest; the output by half a bf16 step
        bound = size * 2.0 ** -7 + p.amax(-1, keepdim=True) * v.abs().sum(0) * 2.0 ** -10 + want.abs() * 2.0 ** -8
        assert bool(((out[:, h].double() - want).abs() <= bound).all()), h
        assert bool(((lse[:, h].double() - torch.logsumexp(s, -1)).abs() <= 1e-4).all()), h
