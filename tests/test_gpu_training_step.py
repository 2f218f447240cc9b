"""A step of training through normed rotary rows: the gradients that it descends along, of its loss, at the weights of each
step, against the formulas in 64 bits and against differences of the loss."""
import pytest
import torch

import decode_attention_02_gb300 as mfa
import norm_reference as norm

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.mark.parametrize("pairing, sections", [("half", (32,)), ("half", (20, 7)), ("adjacent", (16, 8))])
def test_each_step_descends_along_the_gradient_of_its_loss(pairing, sections):
    """loss = sum (y - target)^2 / 2, so dy = y - target."""
    gen = torch.Generator().manual_seed(3)
    op = mfa.NormRope(64, sections, eps=EPS, pairing=pairing)
    x = torch.randn((50, 4, 64), generator=gen)
    pos = torch.arange(50, dtype=torch.int32).expand(len(sections), -1).contiguous()
    target, _ = norm.forward(x, torch.linspace(0.5, 1.5, 64), pos, sections, EPS, pairing=pairing)
    w, aim, args = torch.ones(64), target.float(), (x.to(DEV), pos.to(DEV))

    def loss(weights, rows):
        y, _ = norm.forward(rows, weights, pos, sections, EPS, pairing=pairing)
        return float((y - aim.double()).square().sum() / 2)

    for _ in range(3):
        y, _ = op(args[0], None, w.to(DEV), None, args[1])
        dy = y - aim.to(DEV)
        dx, none, dw, none_w = op.grad(dy, None, args[0], None, w.to(DEV), None, args[1])
        assert none is None and none_w is None
        want_dx, dx_tol, want_dw, dw_tol = norm.gradient(x, dy.cpu(), w, pos, sections, EPS, pairing=pairing)
        for got, want, tol in ((dx, want_dx, dx_tol), (dw, want_dw, dw_tol)):
            assert bool(((got.cpu().double() - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -24).all())
        # Differences of the loss along the gradients: central ones are off by the third derivative, some h^2 of the loss's
        # size over the step's length squared, and 64-bit noise over h; y's fp32 rounding is in dy.
        for got, at in ((dw, w), (dx, x)):
            g = got.cpu().double()
            h = 1e-4 / float(g.norm())
            ahead, behind = ((loss(at.double() + s * h * g, x) if at is w else loss(w, at.double() + s * h * g)) for s in (1, -1))
            slope = (ahead - behind) / (2 * h)
            assert abs(slope - float(g.square().sum())) <= 1e-4 * float(g.square().sum()), (slope, float(g.square().sum()))
        w = w - 0.002 * dw.cpu()
