"""Normed rotary rows: the reference's gradient against differences, and what the library refuses on the host (no GPU)."""
import ctypes

import pytest
import torch

import decode_attention_02_gb300 as mfa
import norm_reference as norm
from decode_attention_02_gb300 import build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return mfa.load_library()


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_the_gradient_formula_against_differences(pairing):
    gen = torch.Generator().manual_seed(1)
    x, dy, v = (torch.randn((3, 2, 12), generator=gen, dtype=torch.float64) for _ in range(3))
    w, vw = (torch.randn((12,), generator=gen, dtype=torch.float64) for _ in range(2))
    pos = torch.randint(-50, 50, (2, 3), generator=gen).to(torch.int32)
    sections, eps, h = (3, 2), 1e-3, 1e-5

    def f(x, w):
        return float((norm.forward(x, w, pos, sections, eps, pairing=pairing)[0] * dy).sum())

    dx, _, dw, _ = norm.gradient(x, dy, w, pos, sections, eps, pairing=pairing)
    # differences: an error of h^2 times third derivatives (of order 10), and 2^-52 / h
    assert abs((f(x + h * v, w) - f(x - h * v, w)) / (2 * h) - float((dx * v).sum())) < 1e-7
    assert abs((f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h) - float((dw * vw).sum())) < 1e-7


def config(**kw):
    a = dict(head_dim=128, rotary_dim=128, num_axes=1, sections=(64, 0, 0, 0), pairing=0, flags=0, theta=1e4, position_scale=1.0)
    a.update(kw)
    a["sections"] = (ctypes.c_int32 * 4)(*a["sections"])
    return mfa.MfaRopeConfig(*a.values())


ROWS = dict(data_in=0x100000, data_out=0x200000, in_stride=512, out_stride=512, heads=4)
GRAD = dict(x=0x100000, dy=0x200000, dx=0x300000, x_stride=512, dy_stride=512, dx_stride=512, heads=4)
KEYS = dict(data_in=0x500000, data_out=0x600000, in_stride=128, out_stride=128, heads=1)
GRAD_KEYS = dict(x=0x500000, dy=0x600000, dx=0x700000, x_stride=128, dy_stride=128, dx_stride=128, heads=1)
INVALID, UNSUPPORTED, WORKSPACE = mfa.MFA_ERR_INVALID_ARG, mfa.MFA_ERR_UNSUPPORTED, mfa.MFA_ERR_WORKSPACE


def run(lib, c=None, q=None, k=None, norm=None, rows=8, dtype=0, table=0x1000, positions=0x2000):
    n = dict(q_weight=0x3000, k_weight=0x4000, weight_dtype=0, eps=1e-6) | (norm or {})
    return lib.mfa_norm_rope_run(c or config(), P(table), P(positions), rows, dtype, mfa.MfaNorm(*n.values()),
                                 mfa.MfaRopeRows(*(ROWS | (q or {})).values()), mfa.MfaRopeRows(*(KEYS | (k or {})).values()), None)


def grad(lib, c=None, q=None, k=None, norm=None, rows=8, dtype=0, table=0x1000, positions=0x2000, dwq=0x8000, dwk=0x9000, ws=0xA000,
         size=8 * 128 * 512):
    n = dict(q_weight=0x3000, k_weight=0x4000, weight_dtype=0, eps=1e-6) | (norm or {})
    return lib.mfa_norm_rope_grad_run(c or config(), P(table), P(positions), rows, dtype, mfa.MfaNorm(*n.values()),
                                      mfa.MfaNormGradRows(*(GRAD | (q or {})).values()),
                                      mfa.MfaNormGradRows(*(GRAD_KEYS | (k or {})).values()), P(dwq), P(dwk), P(ws), size, None)


BOTH = [
    dict(norm=dict(eps=0.0)), dict(norm=dict(eps=-1.0)), dict(norm=dict(eps=float("nan"))), dict(norm=dict(eps=float("inf"))),
    dict(norm=dict(weight_dtype=2)), dict(norm=dict(q_weight=None)), dict(norm=dict(k_weight=None)), dict(norm=dict(q_weight=0x3001)),
    dict(rows=-1), dict(dtype=2), dict(table=None), dict(table=0x1008), dict(positions=None), dict(positions=0x2002),
    dict(q=dict(heads=-1)), dict(q=dict(heads=1 << 30)), dict(c=config(rotary_dim=126)), dict(c=config(theta=0.5)),
]


@pytest.mark.parametrize("kw", BOTH + [
    dict(q=dict(data_in=None)), dict(q=dict(data_out=0x200001)), dict(q=dict(in_stride=511)), dict(k=dict(out_stride=1 << 60)),
    dict(q=dict(data_out=0x100000, out_stride=640)),          # in place with another stride
    dict(q=dict(data_out=0x100002)),                          # over its own input
    dict(k=dict(data_out=0x200000)), dict(k=dict(data_in=0x200100)), dict(k=dict(data_out=0x100100)),
])
def test_refusals(lib, kw):
    assert run(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", BOTH + [
    dict(q=dict(x=None)), dict(q=dict(dy=None)), dict(q=dict(dx=0x300001)), dict(q=dict(dy_stride=511)), dict(k=dict(dy_stride=1 << 60)),
    dict(q=dict(dx=0x100000, dx_stride=640)), dict(q=dict(dx=0x200002)),
    dict(k=dict(dx=0x300000)), dict(k=dict(dx=0x100100)), dict(k=dict(dx=0x200100)), dict(k=dict(dy=0x300100)),
    dict(dwq=0x8001), dict(dwq=0x9000), dict(ws=None), dict(ws=0xA004),
])
def test_refusals_of_the_gradient(lib, kw):
    assert grad(lib, **kw) == INVALID


def test_other_refusals(lib):
    assert run(lib, c=config(head_dim=513, rotary_dim=128)) == UNSUPPORTED
    assert grad(lib, size=8 * 128 * 512 - 1) == WORKSPACE
    assert lib.mfa_norm_rope_run(config(), P(0x1000), P(0x2000), 8, 0, None, mfa.MfaRopeRows(*ROWS.values()), None, None) == INVALID
    assert run(lib, rows=0, table=None, positions=None, norm=dict(q_weight=None, k_weight=None)) == mfa.MFA_OK   # nothing to do
