"""The weights' gradient of normed rotary rows over far more rows than CTAs, with terms of one sign (dy along the output):
what a sum that goes on and on in fp32 loses most from."""
import pytest
import torch

import decode_attention_02_gb300 as mfa
import norm_reference as norm

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5
CTAS, ROW_CTAS, LANES = 304, 456, 288   # at least so many CTAs take the rows; lanes of a CTA's groups


def additions(rows, heads_of_a_slot, slots, ctas):
    """Of fp32 in a row, at most: a thread's own sum (256 terms, or those of 36 rows; then 64 bits), the CTA's slots, 16 and
    32 of the second kernel."""
    chain = -(-rows // ctas) * heads_of_a_slot
    return min(chain, max(256, 36 * heads_of_a_slot)) + slots + 48 + 1


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim, sections, rows, slots, ctas", [
    (64, (32,), 1 << 21, 1, CTAS), (64, (13, 10), 1 << 21, 1, CTAS), (33, (3, 5), 1 << 20, 1, ROW_CTAS), (300, (64,), 1 << 19, 1, 304)])
def test_equal_rows(dim, sections, rows, slots, ctas, dtype, pairing):
    """Each addition rounds the same way.  The terms themselves: 2^-18 of their largest, as elsewhere."""
    gen = torch.Generator().manual_seed(dim)
    x = torch.randn((1, 1, dim), generator=gen).to(dtype)
    w = (1 + torch.randn((dim,), generator=gen) / 4).to(dtype)
    pos = torch.tensor([[7]] * len(sections), dtype=torch.int32)
    op = mfa.NormRope(dim, sections, eps=EPS, pairing=pairing)
    y, _ = op(x.to(DEV), None, w.to(DEV), None, pos.to(DEV))
    _, _, dw, _ = norm.gradient(x, y.cpu(), w, pos, sections, EPS, pairing=pairing)
    xs, ys = x.to(DEV).expand(rows, 1, dim).contiguous(), y.expand(rows, 1, dim).contiguous()
    _, _, got, _ = op.grad(ys, None, xs, None, w.to(DEV), None, pos.to(DEV).expand(-1, rows).contiguous())
    h = (x.double() * norm.scale(x, EPS))[0, 0].abs()
    terms = 2 * y.abs().max().cpu().double() * h * 2.0 ** -18
    tol = rows * (terms + dw.abs() * additions(rows, 1, slots, ctas) * 2.0 ** -24) + rows * dw.abs() * 2.0 ** -24
    off = (got.cpu().double() - rows * dw).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("dim, dtype", [(511, torch.bfloat16), (512, torch.float32), (250, torch.bfloat16)])
def test_equal_rows_of_many_wide_heads(dim, dtype):
    """Heads of up to 512 on every warp of a CTA, each with sums of many terms."""
    heads, rows, sections = (7, 1), 120000, (50,)
    gen = torch.Generator().manual_seed(dim)
    x = [torch.randn((1, n, dim), generator=gen).to(dtype) for n in heads]
    w = [(1 + torch.randn((dim,), generator=gen) / 4).to(dtype) for _ in heads]
    pos = torch.tensor([[7]], dtype=torch.int32)
    op = mfa.NormRope(dim, sections, eps=EPS, pairing="adjacent")
    ww = [t.to(DEV) for t in w]
    y = op(*[t.to(DEV) for t in x], *ww, pos.to(DEV))
    xs, ys = ([t.to(DEV).expand(rows, -1, -1).contiguous() for t in z] for z in (x, y))
    grads = op.grad(*ys, *xs, *ww, pos.to(DEV).expand(-1, rows).contiguous())
    for i in range(2):
        _, _, dw, _ = norm.gradient(x[i], y[i].cpu(), w[i], pos, sections, EPS, pairing="adjacent")
        h = (x[i].double() * norm.scale(x[i], EPS)).abs()
        big = 2 * y[i].cpu().double().abs().amax(-1, keepdim=True)
        own = (norm.turn(y[i].cpu(), pos, sections, 1e4, "adjacent", sign=-1).abs() * h).sum((0, 1))
        tol = rows * ((big * h).sum((0, 1)) * 2.0 ** -18 + own * additions(rows, 1, 8, CTAS) * 2.0 ** -24)
        off = (grads[2 + i].cpu().double() - rows * dw).abs()
        assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("dim, sections, heads, rows, pairing, dtype", [
    (64, (32,), (2, 1), 300000, "half", torch.bfloat16), (256, (44, 42, 42), (64, 1), 22000, "half", torch.bfloat16),
    (33, (3, 5), (9, 2), 70000, "half", torch.bfloat16), (8, (4,), (3, 2), 90000, "adjacent", torch.bfloat16),
    (16, (8,), (40, 0), 90000, "half", torch.float32), (64, (13, 10), (3, 2), 90000, "half", torch.float32),
    (72, (12, 12), (5, 2), 90000, "adjacent", torch.float32), (512, (256,), (1, 1), 80000, "half", torch.bfloat16)])
def test_rows_with_gradients_along_their_outputs(dim, sections, heads, rows, pairing, dtype):
    gen = torch.Generator().manual_seed(rows)
    x = [torch.randn((rows, n, dim), generator=gen).to(dtype) for n in heads]
    w = [(1 + torch.randn((dim,), generator=gen) / 4).to(dtype) for _ in heads]
    pos = torch.randint(0, 100000, (len(sections), rows), generator=gen).to(torch.int32)
    op = mfa.NormRope(dim, sections, eps=EPS, pairing=pairing)
    args = [t.to(DEV) if n else None for t, n in zip(x, heads)] + [t.to(DEV) for t in (*w, pos)]
    y = op(*args)
    grads = op.grad(*y, *args)
    again = op.grad(*y, *args)
    for i, n in enumerate(heads):
        if not n:
            continue
        dx, tol, dw, _ = norm.gradient(x[i], y[i].cpu(), w[i], pos, sections, EPS, pairing=pairing)
        half = torch.finfo(dtype).eps / 2
        assert bool(((grads[i].cpu().double() - dx).abs() <= tol + (dx.abs() + tol) * half).all())
        h = (x[i].double() * norm.scale(x[i], EPS)).abs()
        big = 2 * y[i].cpu().double().abs().amax(-1, keepdim=True)
        terms = (big * h).sum((0, 1)) * 2.0 ** -18
        own = (norm.turn(y[i].cpu(), pos, sections, 1e4, pairing, sign=-1).abs() * h).sum((0, 1))
        tol = terms + own * additions(rows, -(-n // 7), min(n, LANES), CTAS) * 2.0 ** -24
        off = (grads[2 + i].cpu().double() - dw).abs()
        assert bool((off <= tol).all()), float((off / tol).max())
        assert torch.equal(grads[2 + i], again[2 + i]) and torch.equal(grads[i], again[i])
