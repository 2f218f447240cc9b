"""Rotary positions on the GPU against their definition in 64 bits."""
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(rows, heads, dim, axes, seed, dtype, far):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, heads, dim), generator=gen).to(dtype)
    pos = torch.randint(-far, far + 1, (axes, rows), generator=gen).to(torch.int32)
    return x, pos


def check(got, x, want):
    """Two products and a sum of fp32 roundings (3 2^-24), cos and sin of a turn rounded to 24 bits (2 pi 2^-25,
    and 2 ulp of their own): 2^-21 of |a| + |b| in all; and half a step of the output type."""
    half = torch.finfo(got.dtype).eps / 2
    size = x.double().abs().amax(-1, keepdim=True) * 2
    off = (got.cpu().double() - want).abs()
    tol = want.abs() * half + size * 2.0 ** -21
    assert bool((off <= tol).all()), float((off - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dim, sections, heads", [
    (256, (44, 42, 42), (64, 1)), (128, (64,), (64, 4)), (128, (24, 24), (8, 8)), (256, (16, 24, 0, 8), (7, 3)),
    (80, (20, 20), (16, 0)), (72, (12, 12, 12), (3, 5)), (6, (1, 1), (1, 1)), (33, (3, 5, 2, 6), (2, 9)), (512, (200, 56), (5, 1)),
    (511, (1,), (2, 1))])
def test_rope(dim, sections, heads, pairing, dtype):
    for rows, far in ((1, 10), (5, 1 << 20), (67, 2 ** 31 - 1)):
        q, pos = inputs(rows, heads[0], dim, len(sections), rows, dtype, far)
        k, _ = inputs(rows, heads[1], dim, len(sections), rows + 1, dtype, far)
        for kw in (dict(), dict(interleaved=True, theta=5e5), dict(own_spectrum=True, position_scale=0.25)):
            rope = mfa.Rope(dim, sections, pairing=pairing, **kw)
            qo, ko = rope(q.to(DEV), k.to(DEV), pos.to(DEV))
            kw = dict(theta=1e4, pairing=pairing) | kw
            check_far = far < 1 << 30   # fp64 angles of the oracle: 2^-52 of the position
            if check_far:
                check(qo, q, ref.rope(q, pos, sections, **kw))
                check(ko, k, ref.rope(k, pos, sections, **kw))
            # back again: the same angles; each turn within the bound
            back, _ = rope(qo.float(), None, pos.to(DEV), inverse=True)
            size = q.double().abs().amax(-1, keepdim=True) * 2
            tol = size * (2.0 ** -19 + torch.finfo(dtype).eps)
            assert bool(((back.cpu().double() - q.double()).abs() <= tol).all())


def test_positions_at_the_ends_of_their_range():
    """The largest and smallest positions: angles from 64-bit fractions of a turn, against exact integers."""
    rope = mfa.Rope(128, (64,))
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 0, 1]], dtype=torch.int32)
    x = torch.zeros((4, 1, 128))
    x[..., :64] = 1.0
    out, _ = rope(x.to(DEV), None, pos.to(DEV))
    table = mfa.mfa_rope_table(rope.config)
    import math
    for r, p in enumerate(pos[0].tolist()):
        for i in range(64):
            part = (table[i].turns * p % 2 ** 64) / 2 ** 64
            want = (math.cos(2 * math.pi * part), math.sin(2 * math.pi * part))
            assert abs(float(out[r, 0, i]) - want[0]) <= 2.0 ** -20 and abs(float(out[r, 0, i + 64]) - want[1]) <= 2.0 ** -20


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dim, sections", [(128, (30, 10, 8)), (18, (2, 3))])
def test_rope_in_place_and_of_strided_rows(dim, sections, pairing):
    """q and k as columns of one projection, turned in place and into another tensor; the columns between and
    behind stay as they were."""
    rope = mfa.Rope(dim, sections, pairing=pairing)
    gen = torch.Generator().manual_seed(1)
    for dtype in (torch.bfloat16, torch.float32):
        proj = torch.randn((9, 11 * dim), generator=gen).to(dtype)
        pos = torch.randint(0, 5000, (len(sections), 9), generator=gen).to(torch.int32).to(DEV)
        q, k = proj[:, :6 * dim].view(9, 6, dim), proj[:, 7 * dim:9 * dim].view(9, 2, dim)
        wq, wk = rope(q.contiguous().to(DEV), k.contiguous().to(DEV), pos)
        dev = proj.to(DEV)
        dq, dk = dev[:, :6 * dim].view(9, 6, dim), dev[:, 7 * dim:9 * dim].view(9, 2, dim)
        oq, ok = rope(dq, dk, pos)
        assert torch.equal(oq, wq) and torch.equal(ok, wk) and torch.equal(dev.cpu(), proj)
        rope(dq, dk, pos, q_out=dq, k_out=dk)
        assert torch.equal(dq, wq) and torch.equal(dk, wk)
        assert torch.equal(dev[:, 6 * dim:7 * dim].cpu(), proj[:, 6 * dim:7 * dim])
        assert torch.equal(dev[:, 9 * dim:].cpu(), proj[:, 9 * dim:])
        dev = proj.to(DEV)   # only the keys, into columns of another tensor
        into = torch.zeros((9, 3 * dim), dtype=dtype, device=DEV)
        rope(None, dev[:, 7 * dim:9 * dim].view(9, 2, dim), pos, k_out=into[:, dim:].view(9, 2, dim))
        assert torch.equal(into[:, dim:].reshape(9, 2, dim), wk) and bool((into[:, :dim] == 0).all())


def test_rope_gradient():
    """The gradient of sum(w * rope(x)) is the inverse turn of w: against differences (the map is linear) and
    against autograd through the formula."""
    rope = mfa.Rope(64, (10, 6, 8), pairing="adjacent")
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((3, 2, 64), generator=gen)
    w = torch.randn((3, 2, 64), generator=gen)
    pos = torch.randint(0, 3000, (3, 3), generator=gen).to(torch.int32)
    grad, _ = rope(w.to(DEV), None, pos.to(DEV), inverse=True)
    leaf = x.double().requires_grad_()
    turned = ref.rope(torch.eye(64, dtype=torch.float64).view(64, 1, 64), torch.zeros((3, 64), dtype=torch.int32), (10, 6, 8), 1e4,
                      "adjacent")
    assert turned.shape == (64, 1, 64)
    rows = [ref.rope(torch.eye(64, dtype=torch.float64).view(1, 64, 64), pos[:, r:r + 1], (10, 6, 8), 1e4, "adjacent")[0]
            for r in range(3)]   # row r's matrix: e_j turned
    loss = sum((w[r].double() * (leaf[r] @ rows[r])).sum() for r in range(3))
    loss.backward()
    assert bool(((grad.cpu().double() - leaf.grad).abs() <= 2.0 ** -20 * 8).all())
    for r, h, j in ((0, 0, 0), (1, 1, 13), (2, 0, 47), (2, 1, 63)):
        e = torch.zeros_like(x)
        e[r, h, j] = 1.0
        hi, _ = rope((x + e).to(DEV), None, pos.to(DEV))
        lo, _ = rope((x - e).to(DEV), None, pos.to(DEV))
        slope = float(((hi - lo).cpu().double() * w.double()).sum() / 2)
        assert abs(slope - float(grad[r, h, j])) <= 2.0 ** -16


def test_outputs_of_a_call_on_another_stream_stay_until_it_is_done():
    rope, side = mfa.Rope(128, [64]), torch.cuda.Stream()
    q = torch.randn(64, 8, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    rope(q, None, pos, stream=side)   # (loads what is loaded at a first call)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    out, _ = rope(q, None, pos, stream=side)
    used = out.data_ptr()
    del out
    assert torch.empty_like(q).data_ptr() != used or side.query()   # (its memory is free once it is done)
    torch.cuda.synchronize()


def test_rope_repeats_on_any_stream_and_in_a_graph():
    rope = mfa.Rope(256, (64, 32, 32))
    q, pos = inputs(33, 64, 256, 3, 7, torch.bfloat16, 1 << 18)
    q, pos = q.to(DEV), pos.to(DEV)
    want, _ = rope(q, None, pos)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(q)
    rope(q, None, pos, q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope(q, None, pos, q_out=out)
    pos += 17
    graph.replay()
    assert torch.equal(out, rope(q, None, pos)[0])


def test_rope_passes_what_is_not_finite_to_its_pair_alone():
    rope = mfa.Rope(64, (16, 8))
    x, pos = inputs(4, 2, 64, 2, 9, torch.float32, 100)
    want, _ = rope(x.to(DEV), None, pos.to(DEV))
    x[1, 0, 5], x[2, 1, 60] = float("inf"), float("nan")
    got, _ = rope(x.to(DEV), None, pos.to(DEV))
    same = torch.ones(x.shape, dtype=torch.bool)
    same[1, 0, [5, 29]] = False
    same[2, 1, 60] = False      # past the rotated part
    assert torch.equal(got.cpu()[same], want.cpu()[same]) and bool(torch.isnan(got[2, 1, 60]))


def test_rope_checks_its_tensors():
    rope = mfa.Rope(64, (16, 8))
    q = torch.zeros((4, 2, 64), device=DEV)
    pos = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    for args in ((q.half(), None, pos), (q, None, pos.long()), (q, None, pos[:1]), (q[:, :, :32], None, pos),
                 (q.transpose(0, 1), None, pos), (q, q[:3], pos), (q, q.bfloat16(), pos), (q.cpu(), None, pos), (None, None, pos)):
        with pytest.raises(ValueError):
            rope(*args)
    with pytest.raises(ValueError):
        mfa.Rope(64, (16, 8), pairing="other")
    with pytest.raises(ValueError):
        mfa.Rope(64, (1, 1, 1, 1, 1))
    with pytest.raises(mfa.MfaError):
        mfa.Rope(64, (40,))
    empty, _ = rope(q[:0], None, pos[:, :0].contiguous())
    assert empty.shape == (0, 2, 64)
