"""The block-scaled cache's operators and rotary positions in 64 bits, from their definitions.

Tests compare the library with these; nothing here is shared with it.
"""
import math

import torch

PAGE = 64


class Case:
    """Seeded inputs of a block-scaled cache (CPU tensors)."""

    def __init__(self, lens, heads=64, kv_heads=1, dim=256, scale_tokens=64, tokens=1, seed=0, columns=None, spread=1.0,
                 pow2=True, poison=True, q_spread=0.0):
        gen = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.heads, self.kv_heads, self.dim, self.scale_tokens, self.tokens = heads, kv_heads, dim, scale_tokens, tokens
        self.columns = columns or max(1, -(-max(lens + [1]) // PAGE) + 1)
        self.pages = B * self.columns + 2
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)
        self.block_table = torch.randperm(self.pages, generator=gen)[:B * self.columns].to(torch.int32).view(B, -1).contiguous()
        q = torch.randn((B * tokens, heads, dim), generator=gen)
        if q_spread:   # heads of different magnitudes
            q = q * torch.exp2((torch.rand((B * tokens, heads, 1), generator=gen) * 2 - 1) * q_spread)
        self.q = q.bfloat16()
        for name in ("k", "v"):
            x = torch.randn((self.pages, kv_heads, PAGE // scale_tokens, scale_tokens, dim), generator=gen)
            x = x * torch.exp2((torch.rand((self.pages, kv_heads, PAGE // scale_tokens, 1, 1), generator=gen) * 2 - 1) * spread)
            a = x.abs().amax((3, 4))
            s = torch.exp2(torch.ceil(torch.log2(a / 448))) if pow2 else a / 448
            c = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            setattr(self, name + "_cache", c.view(self.pages, kv_heads, PAGE, dim).contiguous())
            setattr(self, name + "_scale", s.contiguous())
        if poison:   # what no token names holds NaN
            used = torch.zeros((self.pages, PAGE), dtype=torch.bool)
            for b, L in enumerate(lens):
                for j in range(-(-L // PAGE)):
                    used[self.block_table[b, j], :min(PAGE, L - PAGE * j)] = True
            for name in ("k", "v"):
                cache, scale = getattr(self, name + "_cache"), getattr(self, name + "_scale")
                cache.copy_(torch.where(used[:, None, :, None], cache, torch.tensor(0x7F, dtype=torch.uint8)))
                live = used.view(self.pages, PAGE // scale_tokens, scale_tokens).any(-1)
                scale.copy_(torch.where(live[:, None], scale, torch.tensor(float("nan"))))

    def rows(self, name, b, L):
        """[kv_heads, L, dim] values of the sequence's first L tokens, and [kv_heads, L] scales."""
        cache, scale = getattr(self, name + "_cache"), getattr(self, name + "_scale")
        idx = self.block_table[b, :-(-L // PAGE)].long()
        s = scale[idx].double().repeat_interleave(self.scale_tokens, 2).transpose(0, 1).reshape(self.kv_heads, -1)[:, :L]
        x = cache[idx].view(torch.float8_e4m3fn).double().transpose(0, 1).reshape(self.kv_heads, -1, self.dim)[:, :L]
        return x * s[..., None], s


def decode(case, softmax_scale=None):
    """(out, lse, tol, lse_tol): fp64 results, and how far the library's fp32 result may be off.

    The bound counts the roundings of the e4m3 path, per output element:
    - scores: q is split into two e4m3 parts, off by at most 2^-16 of its row's largest element
      (where an element is under 2^-9 of it); the products are exact and their sum, the scale's
      product and the subtraction of the reference are in fp32: (dim + 4) 2^-23 sum |q k|.
      A score off by e changes a weight and the sum of weights by at most e^(2 e) - 1.
    - weights: rounded to f16 (2^-11), then split into two e4m3 parts: 2^-8 of what is left (a part is
      off by 2^-4 of itself), or the half step 2^-10 of e4m3's smallest numbers where 16 times that
      (relative to the row's largest weight times its value scale, at least) is small, and never
      more than itself.  The two add up: where the half step is the larger, the f16 rounding of the
      weight comes on top of it.
    - fp32 sums: 2^-18.
    """
    B, T, H, G, d = len(case.seq_lens), case.tokens, case.heads, case.kv_heads, case.dim
    scale = d ** -0.5 if softmax_scale is None else softmax_scale
    out = torch.zeros((B * T, H, d), dtype=torch.float64)
    lse = torch.full((B * T, H), float("-inf"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse_tol = torch.zeros_like(lse)
    for b, L in enumerate(case.seq_lens.tolist()):
        if L == 0:
            continue
        k, _ = case.rows("k", b, L)
        v, sv = case.rows("v", b, L)
        for i in range(T):
            n = L - (T - 1) + i
            if n <= 0:
                continue
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                q = case.q[b * T + i, hs].double()
                s = scale * q @ k[g, :n].T
                m = s.amax(-1, keepdim=True)
                p = torch.exp(s - m)
                l = p.sum(-1, keepdim=True)
                w = p / l
                out[b * T + i, hs] = w @ v[g, :n]
                lse[b * T + i, hs] = (m + torch.log(l)).squeeze(-1)
                qmax = q.abs().amax(-1, keepdim=True)
                small = (q.abs() < qmax * 2.0 ** -8) * qmax * 2.0 ** -16
                e = (scale * small @ k[g, :n].abs().T + (d + 4) * 2.0 ** -23 * scale * q.abs() @ k[g, :n].abs().T).amax(-1, keepdim=True)
                e = e + 2.0 ** -22 * s.abs().amax(-1, keepdim=True)
                shift = torch.expm1(2 * e)
                step = 2.0 ** -14 * (p * sv[g, :n]).amax(-1, keepdim=True) / sv[g, :n] / l     # e4m3's half step, as a weight
                dw = torch.minimum(torch.maximum(2.0 ** -8 * w, step), w) + 2.0 ** -10 * w
                tol[b * T + i, hs] = (dw + (shift + 2.0 ** -18) * w) @ v[g, :n].abs() + 1e-30
                lse_tol[b * T + i, hs] = (e + 2.0 ** -18 + 2.0 ** -23 * lse[b * T + i, hs, None].abs()).squeeze(-1)
    return out, lse, tol, lse_tol


def append(cache, scale, block_table, positions, new, offsets, scale_tokens, capacity):
    """The append's result for one pool: (codes uint8, scales fp32), block by block."""
    codes, scales = cache.clone(), scale.clone()
    G = cache.shape[1]
    for b, t0 in enumerate(positions.tolist()):
        r0, r1 = int(offsets[b]), int(offsets[b + 1])
        if t0 < 0:
            continue
        end = min(t0 + r1 - r0, capacity)
        t = t0
        while t < end:
            first = t // scale_tokens * scale_tokens
            stop = min(end, first + scale_tokens)
            page = int(block_table[b, t // PAGE])
            if not 0 <= page < cache.shape[0]:
                t = stop
                continue
            lo, hi, sub = t % PAGE, t % PAGE + stop - t, first % PAGE // scale_tokens
            for g in range(G):
                x = new[r0 + t - t0:r0 + stop - t0, g].double()
                fin = x[torch.isfinite(x)]
                a = float(fin.abs().max()) if fin.numel() else 0.0
                e = -126
                while a > 448 * 2.0 ** e:
                    e += 1
                s = 2.0 ** e
                if t > first:
                    old = float(scales[page, g, sub])
                    s = max(s, old)
                    if s > old:
                        was = codes[page, g, first % PAGE:lo].view(torch.float8_e4m3fn).float()
                        ratio = torch.tensor(old, dtype=torch.float32) / torch.tensor(s, dtype=torch.float32)
                        codes[page, g, first % PAGE:lo] = (was * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
                scales[page, g, sub] = s
                # the quotient in fp32, infinities saturated as the cast does not
                y = (x.float() / torch.tensor(s, dtype=torch.float32)).clamp(-448, 448)
                codes[page, g, lo:hi] = y.to(torch.float8_e4m3fn).view(torch.uint8)
            t = stop
    return codes, scales


def rope_axes(sections, interleaved):
    """The axis of each pair."""
    left, axes, a = list(sections), [], 0
    while any(left):
        if interleaved:
            if left[a]:
                axes.append(a)
                left[a] -= 1
            a = (a + 1) % len(left)
        else:
            a = next(i for i, n in enumerate(left) if n)
            axes.append(a)
            left[a] -= 1
    return axes


def rope(x, positions, sections, theta, pairing, interleaved=False, own_spectrum=False, position_scale=1.0, sign=1):
    """x [rows, heads, d] turned, in fp64."""
    pairs = sum(sections)
    y = x.double().clone()
    seen = [0] * len(sections)
    for i, a in enumerate(rope_axes(sections, interleaved)):
        power = seen[a] / sections[a] if own_spectrum else i / pairs
        seen[a] += 1
        w = sign * positions[a].double() * position_scale * math.pow(theta, -power)
        j, k = (i, i + pairs) if pairing == "half" else (2 * i, 2 * i + 1)
        c, s = torch.cos(w)[:, None], torch.sin(w)[:, None]
        p, q = x[..., j].double(), x[..., k].double()
        y[..., j], y[..., k] = p * c - q * s, q * c + p * s
    return y
