"""Attention over a block-scaled cache where each new token sees tokens of its own, in 64 bits from the definition.

Tests of windowed decodes and of trees compare the library with this; nothing here is shared with it.
"""
import torch

PAGE = 64


def window_seen(L, T, window, sinks):
    """[T, L]: what the last T of L tokens see through a window, with first tokens that stay visible."""
    t, p = torch.arange(L), (L - T + torch.arange(T))[:, None]
    return (t <= p) & ((t < sinks) | (t > p - window))


def tree_seen(L, T, masks):
    """[T, L]: the tokens before the tree's T, and those of the tree that a node's mask names."""
    node = torch.arange(L) - (L - T)
    bits = torch.tensor([[m >> j & 1 for j in range(T)] for m in masks], dtype=torch.bool).reshape(T, T)
    return (node < 0) | bits[:, node.clamp(min=0)]


def rows(case, name, b, L):
    """[kv_heads, L, dim] values and [kv_heads, L] scales of a sequence's first L tokens (ids outside the pool: any page)."""
    cache, scale = getattr(case, name + "_cache"), getattr(case, name + "_scale")
    idx = case.block_table[b, :-(-L // PAGE)].long()
    idx = torch.where((idx >= 0) & (idx < cache.shape[0]), idx, 0)
    s = scale[idx].double().repeat_interleave(case.scale_tokens, 2).transpose(0, 1).reshape(case.kv_heads, -1)[:, :L]
    x = cache[idx].view(torch.float8_e4m3fn).double().transpose(0, 1).reshape(case.kv_heads, -1, case.dim)[:, :L]
    return x * s[..., None], s


def decode(case, seen, out_rows, weight_bound, softmax_scale=None):
    """(out, lse, tol, lse_tol) of the new tokens in fp64, and how far the library's fp32 result may be off.

    ``seen(b, L)``: bool [out_rows, L].  The bound counts, per output element: scores and sums as the
    decode of whole sequences has them (q in two e4m3 parts: 2^-16 of its row's largest where an element is
    under 2^-9 of it; fp32 products and sums: (dim + 4) 2^-23 sum |q k|), and the rounding of a weight:
    ``weight_bound(w, p, sv, l, the tokens)``.  fp32 sums: 2^-18.
    """
    B, T, H, G, d = len(case.seq_lens), out_rows, case.heads, case.kv_heads, case.dim
    scale = d ** -0.5 if softmax_scale is None else softmax_scale
    out = torch.zeros((B * T, H, d), dtype=torch.float64)
    lse = torch.full((B * T, H), float("-inf"), dtype=torch.float64)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, L in enumerate(case.seq_lens.tolist()):
        if L == 0:
            continue
        mask = seen(b, L)
        k, _ = rows(case, "k", b, L)
        v, sv = rows(case, "v", b, L)
        for i in range(T):
            see = mask[i]
            if not bool(see.any()):
                continue
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                q, kk, vv, ss = case.q[b * T + i, hs].double(), k[g][see], v[g][see], sv[g][see]
                s = scale * q @ kk.T
                m = s.amax(-1, keepdim=True)
                p = torch.exp(s - m)
                l = p.sum(-1, keepdim=True)
                w = p / l
                out[b * T + i, hs] = w @ vv
                lse[b * T + i, hs] = (m + torch.log(l)).squeeze(-1)
                qmax = q.abs().amax(-1, keepdim=True)
                small = (q.abs() < qmax * 2.0 ** -8) * qmax * 2.0 ** -16
                e = (scale * small @ kk.abs().T + (d + 4) * 2.0 ** -23 * scale * q.abs() @ kk.abs().T).amax(-1, keepdim=True)
                e = e + 2.0 ** -22 * s.abs().amax(-1, keepdim=True)
                dw = weight_bound(w, p, ss, l, see.nonzero().flatten())
                tol[b * T + i, hs] = (dw + (torch.expm1(2 * e) + 2.0 ** -18) * w) @ vv.abs() + 1e-30
                lse_tol[b * T + i, hs] = (e + 2.0 ** -18 + 2.0 ** -23 * lse[b * T + i, hs, None].abs()).squeeze(-1)
    return out, lse, tol, lse_tol


def two_e4m3(w, p, sv, l, t):
    """A weight rounded to f16 (2^-11) and split into two e4m3 parts: 2^-8 of it, or the half step of e4m3's smallest
    numbers, 2^-14 of the row's largest weight times value scale, and never more than itself; and 2^-10 for the f16."""
    top = (p * sv).amax(-1, keepdim=True)
    return torch.minimum(torch.maximum(2.0 ** -8 * w, 2.0 ** -14 * top / sv / l), w) + 2.0 ** -10 * w


def e4m3_and_e5m2(w, p, sv, l, t):
    """A weight times its value scale, P, rounded to f16 (2^-11) and split into an e4m3 part and an e5m2 one of what is
    left, where the largest P of its 128 tokens is 2^-3 at least: 2^-7 of itself (2^-4 by 2^-3); under 2^-6, where the
    first part's half step is 2^-10, 2^-3 of that or of itself; 2^-17, the second part's smallest half step, or itself.
    (References reach 24 under the highest, whose P is 2^8.75 at most: 2^-40 of the row's largest beside it.)"""
    P = p * sv
    top = torch.zeros_like(P)
    for j in t.div(128, rounding_mode="floor").unique():
        at = t.div(128, rounding_mode="floor") == j
        top[:, at] = P[:, at].amax(-1, keepdim=True)
    top = torch.maximum(top, P.amax(-1, keepdim=True) * 2.0 ** -27)
    split = torch.maximum(2.0 ** -7 * P, torch.minimum(2.0 ** -3 * P, 2.0 ** -10 * top)) + torch.minimum(P, 2.0 ** -14 * top)
    return split / sv / l + 2.0 ** -10 * w


def check(out, lse, expect):
    """out (bf16: half a step, 2^-8 of the value, more) and lse within the derived bounds; rows that see nothing
    zeros and -inf."""
    want, want_lse, tol, lse_tol = expect
    got = out.cpu().double()
    if out.dtype is torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(((got - want).abs() - tol).max()))
    gl = lse.cpu().double()
    empty = torch.isinf(want_lse)
    assert torch.equal(gl[empty], want_lse[empty])
    off = (gl - want_lse).abs()[~empty]
    assert bool((off <= lse_tol[~empty]).all()), float((off - lse_tol[~empty]).max())
    assert bool((got.reshape(lse.shape + (-1,))[empty] == 0).all())


def hide(case, keep, pages_too=True):
    """NaN codes and scales for the tokens outside keep(b, L) (bool [L]), and ids outside the pool for pages that
    hold none of them."""
    for b, L in enumerate(case.seq_lens.tolist()):
        k = torch.zeros(case.columns * PAGE, dtype=torch.bool)
        k[:L] = keep(b, L)
        for j in range(case.columns):
            held, page = k[j * PAGE:(j + 1) * PAGE], int(case.block_table[b, j])
            for name in ("k", "v"):
                getattr(case, name + "_cache")[page][:, ~held] = 0x7F
                blocks = held.view(-1, case.scale_tokens).any(-1)
                getattr(case, name + "_scale")[page][:, ~blocks] = float("nan")
            if pages_too and not bool(held.any()):
                case.block_table[b, j] = (-1, 1 << 30)[j % 2]
