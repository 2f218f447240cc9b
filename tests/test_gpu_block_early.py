"""Block decode that reads its lengths before the preceding kernel is done (MFA_PLAN_EARLY_METADATA), on the GPU."""
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa
from test_gpu_block import DEV, GQA, MFA, SINGLE, TWELVE, WAYS, check, decoder, device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way, lens, shape, kw, ctas", [
    ("clusters", [300] * 130, MFA, dict(), 0),
    ("clusters", [1024] * 20, MFA, dict(), 0),
    ("even", [900, 1, 0, 200], MFA, dict(tokens=3), 12),
    ("even", [9000, 100, 0, 3000], GQA, dict(tokens=2), 0),
    ("cost", [700] * 200, SINGLE, dict(), 0),
    ("cost", [100, 3000, 700, 0, 1], TWELVE, dict(tokens=2), 7),
])
def test_early_lengths_in_every_way(way, lens, shape, kw, ctas):
    """Behind kernels that write q, the new rows and the outputs' memory, one after another without a pause."""
    c = ref.Case(lens, **shape, **kw, scale_tokens=32, seed=len(lens))
    early = decoder(c, force_ctas=ctas, flags=mfa.MFA_PLAN_EARLY_METADATA, out_dtype=mfa.MFA_OUT_FP32)
    assert early.plan.flags == mfa.MFA_PLAN_EARLY_METADATA | WAYS[way]
    d = device(c)
    want = ref.decode(c)
    q, results = torch.empty_like(d[0]), []
    no_rows = torch.full((len(lens),), -1, dtype=torch.int32, device=DEV)
    new = torch.zeros((len(lens) * c.tokens, c.kv_heads, c.dim), dtype=torch.bfloat16, device=DEV)
    rope = mfa.Rope(c.dim, (c.dim // 2,))
    still = torch.zeros((1, q.shape[0]), dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    for _ in range(4):
        q.zero_()
        rope(d[0], None, still, q_out=q)                 # position 0: a copy, by a kernel that lets the next one start
        early.append(new, new, no_rows, d[5], *d[1:5])
        results.append(early(q, *d[1:]))
    torch.cuda.synchronize()
    for out, lse in results:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    check(c, *results[0], want)
    assert mfa.mfa_read_device_status(early.workspace) == 0


def test_early_lengths_in_a_graph():
    c = ref.Case([700, 64, 1500], **GQA, tokens=2, seed=13)
    d, dec = device(c), decoder(c, lens=None, flags=mfa.MFA_PLAN_EARLY_METADATA, out_dtype=mfa.MFA_OUT_FP32)
    want = dec(*d)
    out, lse = (torch.zeros_like(x) for x in want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            dec(*d, out=out, lse=lse)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    check(c, out, lse)
