"""Each weight of a tree decode by itself: token t's values are a one at element t, so that an output element is a weight."""
import pytest
import torch

import decode_attention_02_gb300 as mfa
from test_tree_rounding import stated

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dim, block", [(128, 16), (256, 64)])
@pytest.mark.parametrize("lowest", [1.0, 9.0, 13.0, 16.0, 20.0])
def test_each_weight(dim, block, lowest):
    """Scores that go down to `lowest` powers of two under the largest, which stands alone or not."""
    L = 128
    for crowd in (1, 40):
        gen = torch.Generator().manual_seed(int(lowest) + crowd)
        k = torch.zeros((2, 1, 64, dim))
        score = torch.rand((2, 64), generator=gen) * 448
        score.view(-1)[torch.randperm(L, generator=gen)[:crowd]] = 448
        k[:, 0, :, 0] = score
        codes = k.to(torch.float8_e4m3fn)
        v = torch.zeros((2, 1, 64, dim))
        v.view(L, dim)[torch.arange(L), torch.arange(L) % dim] = 1
        q = torch.zeros((1, 1, dim), dtype=torch.bfloat16)
        q[..., 0] = 1
        scale = lowest * torch.log(torch.tensor(2.0, dtype=torch.float64)).item() / 448
        dec = mfa.TreeDecoder(1, 2, 2, 1, num_q_heads=1, num_kv_heads=1, head_dim=dim, scale_tokens=block, softmax_scale=scale,
                              host_seq_lens=[L], out_dtype=mfa.MFA_OUT_FP32, flags=mfa.MFA_PLAN_CHECK)
        one = torch.ones((2, 1, 64 // block), device=DEV)
        out, lse = dec(q.to(DEV), codes.view(torch.uint8).to(DEV), v.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV), one, one.clone(),
                       torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), torch.tensor([L], dtype=torch.int32, device=DEV),
                       torch.ones((1, 1), dtype=torch.int64, device=DEV))
        # (the softmax scale goes to the library in fp32)
        s = codes.double().view(L, dim)[:, 0] * float(torch.tensor(scale, dtype=torch.float32))
        w = torch.softmax(s, 0)
        got = out.cpu().double().view(dim)[:L]
        # scores: fp32 products, the scale in powers of two and the reference, 2^-22 of 20 powers of two; sums 2^-18
        tol = stated(w, w.max()) + w * 2.0 ** -16
        assert bool(((got - w).abs() <= tol).all()), float(((got - w).abs() / tol).max())
        assert abs(float(lse) - float(torch.logsumexp(s, 0))) < 2.0 ** -18
