"""Normed rotary rows and their gradient on the GPU, against their definitions in 64 bits."""
import pytest
import torch

import decode_attention_02_gb300 as mfa
import norm_reference as norm

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5

SHAPES = [(256, (44, 42, 42), (64, 1)), (128, (64,), (64, 4)), (128, (24, 24), (8, 8)), (256, (16, 24, 0, 8), (7, 3)),
          (80, (20, 20), (16, 0)), (72, (12, 12, 12), (3, 5)), (6, (1, 1), (1, 1)), (33, (3, 5, 2, 6), (2, 9)),
          (512, (200, 56), (5, 1)), (512, (8,), (2, 3)), (511, (1,), (2, 1)), (8, (4,), (40, 90)), (256, (128,), (0, 70)),
          (16, (8,), (130, 1)), (32, (4,), (1, 200))]


def inputs(rows, heads, dim, axes, seed, dtype, weight_type=None):
    gen = torch.Generator().manual_seed(seed)
    x = [torch.randn((rows, n, dim), generator=gen) * torch.exp2(torch.randint(-6, 7, (rows, n, 1), generator=gen)) for n in heads]
    dy = [torch.randn((rows, n, dim), generator=gen) for n in heads]
    w = [(1 + torch.randn((dim,), generator=gen) / 4).to(weight_type or dtype) for _ in heads]
    pos = torch.randint(-100000, 100000, (axes, rows), generator=gen).to(torch.int32)
    return [t.to(dtype) for t in x], [t.to(dtype) for t in dy], w, pos


def rounded(got, want, tol):
    """Half a step of the output's type beside the bound."""
    half = torch.finfo(got.dtype).eps / 2
    off = (got.cpu().double() - want).abs()
    bound = tol + (want.abs() + tol) * half
    assert bool((off <= bound).all()), (float((off - bound).max()), (off > bound).nonzero()[:4].tolist())


@pytest.mark.parametrize("dtype, weight_type", [(torch.bfloat16, None), (torch.float32, None), (torch.bfloat16, torch.float32),
                                                (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dim, sections, heads", SHAPES)
def test_forward_and_gradient(dim, sections, heads, pairing, dtype, weight_type):
    for rows in (1, 5, 67):
        x, dy, w, pos = inputs(rows, heads, dim, len(sections), rows, dtype, weight_type)
        for kw in (dict(), dict(interleaved=True, theta=5e5), dict(own_spectrum=True, position_scale=0.25)):
            op = mfa.NormRope(dim, sections, eps=EPS, pairing=pairing, **kw)
            kw = dict(theta=1e4, pairing=pairing) | kw
            d = [t.to(DEV) if n else None for t, n in zip(x, heads)]
            dd = [t.to(DEV) if n else None for t, n in zip(dy, heads)]
            ww = [t.to(DEV) for t in w]
            out = op(*d, *ww, pos.to(DEV))
            grads = op.grad(*dd, *d, *ww, pos.to(DEV))
            for i, n in enumerate(heads):
                if not n:
                    assert out[i] is None and grads[i] is None and grads[2 + i] is None
                    continue
                rounded(out[i], *norm.forward(x[i], w[i], pos, sections, EPS, **kw))
                dx, tol, dw, dw_tol = norm.gradient(x[i], dy[i], w[i], pos, sections, EPS, **kw)
                rounded(grads[i], dx, tol)
                rounded(grads[2 + i], dw, dw_tol)
                assert grads[2 + i].dtype is torch.float32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dim, sections, heads", [(256, (50,), (24, 2)), (128, (1,), (64, 4)), (64, (13, 10), (5, 3)), (256, (127,), (3, 1)),
                                                  (512, (255,), (2, 1)), (8, (3,), (40, 2)), (72, (30, 5), (9, 9)), (256, (2, 3, 4, 5), (1, 0))])
def test_pairs_that_are_no_eights(dim, sections, heads, pairing, dtype):
    """(Adjacent ones: a vector of eight elements holds turned pairs and others.)"""
    for rows in (3, 500):
        x, dy, w, pos = inputs(rows, heads, dim, len(sections), rows, dtype)
        op = mfa.NormRope(dim, sections, eps=EPS, pairing=pairing)
        d, dd = ([t.to(DEV) if n else None for t, n in zip(y, heads)] for y in (x, dy))
        ww = [t.to(DEV) for t in w]
        out = op(*d, *ww, pos.to(DEV))
        grads = op.grad(*dd, *d, *ww, pos.to(DEV))
        for i in range(2 if heads[1] else 1):
            rounded(out[i], *norm.forward(x[i], w[i], pos, sections, EPS, theta=1e4, pairing=pairing))
            dx, tol, dw, dw_tol = norm.gradient(x[i], dy[i], w[i], pos, sections, EPS, theta=1e4, pairing=pairing)
            rounded(grads[i], dx, tol)
            rounded(grads[2 + i], dw, dw_tol)


@pytest.mark.parametrize("dim, sections, heads", [(256, (128,), (64, 1)), (128, (24, 24), (40, 8)), (33, (3, 5), (3, 2))])
def test_many_rows(dim, sections, heads):
    """More rows than CTAs: their sums go on over rows.  The gradient twice gives the same bits."""
    x, dy, w, pos = inputs(1013, heads, dim, len(sections), 3, torch.bfloat16)
    op = mfa.NormRope(dim, sections, eps=EPS)
    args = [t.to(DEV) for t in (*dy, *x, *w, pos)]
    grads = op.grad(*args)
    for i in range(2):
        dx, tol, dw, dw_tol = norm.gradient(x[i], dy[i], w[i], pos, sections, EPS)
        rounded(grads[i], dx, tol)
        rounded(grads[2 + i], dw, dw_tol)
    for a, b in zip(grads, op.grad(*args)):
        assert torch.equal(a, b)


def test_rows_of_zeros_and_far_magnitudes():
    """A zero head stays zero and has the gradient of eps alone; heads of 1e-15 and 1e15."""
    x, dy, w, pos = inputs(6, (3, 1), 128, 1, 5, torch.float32)
    x[0][0] = 0
    x[0][1] *= 1e-15
    x[0][2] *= 1e15
    op = mfa.NormRope(128, (64,), eps=EPS)
    out = op(*[t.to(DEV) for t in (*x, *w, pos)])
    grads = op.grad(*[t.to(DEV) for t in (*dy, *x, *w, pos)])
    assert bool((out[0][0] == 0).all())
    rounded(out[0], *norm.forward(x[0], w[0], pos, (64,), EPS))
    dx, tol, dw, dw_tol = norm.gradient(x[0], dy[0], w[0], pos, (64,), EPS)
    rounded(grads[0], dx, tol)
    rounded(grads[2], dw, dw_tol)


def test_a_bad_head_spoils_its_own_rows_alone():
    x, _, w, pos = inputs(4, (4, 2), 128, 1, 5, torch.bfloat16)
    op = mfa.NormRope(128, (64,))
    good = op(*[t.to(DEV) for t in (*x, *w, pos)])
    x[0][1, 2, 77] = float("nan")
    x[1][3, 0, 5] = float("inf")
    bad = op(*[t.to(DEV) for t in (*x, *w, pos)])
    same = [a == b for a, b in zip(good, bad)]
    same[0][1, 2] = same[1][3, 0] = True
    assert all(bool(s.all()) for s in same)


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dim, sections", [(128, (30, 10, 8)), (18, (2, 3))])
def test_in_place_and_strided(dim, sections, pairing):
    """q and k as columns of one projection: turned in place, into another tensor, gradients over dy and over x; the
    columns between and behind stay as they were."""
    op = mfa.NormRope(dim, sections, eps=EPS, pairing=pairing)
    gen = torch.Generator().manual_seed(1)
    for dtype in (torch.bfloat16, torch.float32):
        x, dy, w, pos = inputs(9, (6, 2), dim, len(sections), 2, dtype)
        pos, w = pos.to(DEV), [t.to(DEV) for t in w]
        d = [t.to(DEV) for t in x]
        plain, plain_grads = op(*d, *w, pos), op.grad(*[t.to(DEV) for t in dy], *d, *w, pos)

        def columns(a, b):
            t = torch.randn((9, 11 * dim), generator=gen).to(dtype).to(DEV)
            q, k = t[:, :6 * dim].view(9, 6, dim), t[:, 7 * dim:9 * dim].view(9, 2, dim)
            q.copy_(a)
            k.copy_(b)
            rest = torch.cat([t[:, 6 * dim:7 * dim], t[:, 9 * dim:]], 1).clone()
            return t, q, k, lambda: torch.equal(torch.cat([t[:, 6 * dim:7 * dim], t[:, 9 * dim:]], 1), rest)

        t, q, k, untouched = columns(*x)
        out = op(q, k, *w, pos)
        assert all(torch.equal(a, b) for a, b in zip(out, plain)) and torch.equal(q, d[0])
        g, gq, gk, g_untouched = columns(*dy)
        grads = op.grad(gq, gk, q, k, *w, pos, q_grad=gq, k_grad=gk)
        assert all(torch.equal(a, b) for a, b in zip(grads, plain_grads)) and g_untouched()
        g, gq, gk, _ = columns(*dy)
        t2, q2, k2, untouched2 = columns(*x)
        grads = op.grad(gq, gk, q2, k2, *w, pos, q_grad=q2, k_grad=k2)
        assert all(torch.equal(a, b) for a, b in zip(grads, plain_grads)) and untouched2() and torch.equal(gq, dy[0].to(DEV))
        op(q, k, *w, pos, q_out=q, k_out=k)
        assert torch.equal(q, plain[0]) and torch.equal(k, plain[1]) and untouched()


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dim, sections", [(256, (50,)), (128, (3, 2)), (248, (100, 23)), (64, (31,))])
def test_in_place_with_pairs_that_are_no_eights(dim, sections, pairing):
    """(Half pairing: lanes read what other lanes of the head have copied.)"""
    test_in_place_and_strided(dim, sections, pairing)


def test_gradient_against_differences():
    """<dx, v> + <dw, vw> against a central difference of the call itself, in fp32: outputs off by 2^-18 of about 4 each,
    n of them at random signs, over 2 h; and h^2 / 6 of a third derivative of at most 8 sum |dy| |v|^3."""
    op = mfa.NormRope(128, (40, 24), eps=EPS, pairing="adjacent")
    gen = torch.Generator().manual_seed(4)
    x, dy, v = (torch.randn((5, 4, 128), generator=gen) for _ in range(3))
    w, vw = 1 + torch.randn((128,), generator=gen) / 4, torch.randn((128,), generator=gen) / 4
    pos = torch.randint(0, 5000, (2, 5), generator=gen).to(torch.int32).to(DEV)
    h = 2.0 ** -7

    def f(s):
        out, _ = op((x + s * v).to(DEV), None, (w + s * vw).to(DEV), None, pos)
        return float((out.cpu().double() * dy.double()).sum())

    dx, _, dw, _ = op.grad(dy.to(DEV), None, x.to(DEV), None, w.to(DEV), None, pos)
    want = float((dx.cpu().double() * v.double()).sum() + (dw.cpu().double() * vw.double()).sum())
    n = x.numel()
    bound = 4 * 2.0 ** -18 * n ** 0.5 * 4 / (2 * h) + h * h / 6 * 8 * float((dy.abs() * v.abs() ** 3).sum())
    assert abs((f(h) - f(-h)) / (2 * h) - want) <= bound


def test_no_rows_and_refusals():
    op = mfa.NormRope(128, (64,))
    w = torch.ones((128,), dtype=torch.bfloat16, device=DEV)
    none, pos = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=DEV), torch.empty((1, 0), dtype=torch.int32, device=DEV)
    out = op(none, None, w, None, pos)
    assert out[0].shape == none.shape and out[1] is None
    dx, _, dw, _ = op.grad(none, None, none, None, w, None, pos)
    assert dx.shape == none.shape and bool((dw == 0).all())
    x, pos = torch.randn((3, 4, 128), device=DEV).bfloat16(), torch.zeros((1, 3), dtype=torch.int32, device=DEV)
    for args in ((None, None, w, w, pos), (x, None, None, None, pos), (x, x, w, None, pos), (x, None, w[:64], None, pos),
                 (x, None, w.half(), None, pos), (x.half(), None, w, None, pos), (x, x, w, w.float(), pos), (x, None, w.cpu(), None, pos),
                 (x, None, w, None, pos[:, :2]), (x, None, w, None, pos.long()), (x[..., :64], None, w, None, pos),
                 (x.transpose(0, 1), None, w, None, pos), (x, x.float(), w, w, pos), (x[:, ::2], None, w, None, pos)):
        with pytest.raises(ValueError):
            op(*args)
    with pytest.raises(ValueError):
        op.grad(None, None, x, None, w, None, pos)
    with pytest.raises(ValueError):
        op.grad(x[:2], None, x, None, w, None, pos)
    with pytest.raises(ValueError):
        op.grad(x.float(), None, x, None, w, None, pos)
    with pytest.raises(mfa.MfaError):
        op(x, x, w, w, pos, q_out=x, k_out=x)
    with pytest.raises(mfa.MfaError):
        mfa.NormRope(128, (64,), eps=0.0)(x, None, w, None, pos)


def test_in_a_graph_and_on_another_stream():
    x, dy, w, pos = inputs(33, (64, 1), 256, 1, 9, torch.bfloat16)
    op = mfa.NormRope(256, (128,), eps=EPS)
    args = [t.to(DEV) for t in (*dy, *x, *w, pos)]
    want, want_grads = op(*args[2:]), op.grad(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, grads = op(*args[2:], stream=side), op.grad(*args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *grads), (*want, *want_grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, grads = op(*args[2:]), op.grad(*args)
    for _ in range(2):
        for t in (*got, *grads):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *grads), (*want, *want_grads)))
