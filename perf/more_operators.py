"""Serving and training operators next to the block-scaled 8-bit KV cache, as measured cases.

Three operators, in the order in which a step of a model with normed queries and keys uses them:

``norm``    each head of the queries and of the new keys divided by its root mean square, times a
            weight for each element, then turned by its position, in one pass; and its gradient
            (``grad``), which training takes;
``window``  attention of 1 to 4 new tokens a sequence that see the last ``window`` tokens and the
            first ``sinks`` ones of the cache;
``tree``    attention of a tree of drafted tokens: each sees the cache before the tree, and of the
            tree the nodes that its mask names (its ancestors and itself).

``run`` computes them in elementary torch operations where ``own`` is false, and through the
package's entry points where it is true.

The cache: codes uint8 [pages, kv heads, 64, width], scales fp32 [pages, kv heads, 64 / block];
a value is e4m3(code) * scale.  ``block_table`` int32 [sequences, columns] names the pages.
"""
import math

import torch

own = False

PAGE = 64
E4M3_MAX = 448.0
EPS = 1e-6
MFA = dict(heads=64, kv_heads=1, width=256)     # one shared key head and one shared value head
GQA = dict(heads=64, kv_heads=4, width=128)     # grouped heads


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # the query heads and the new key of one decode step
        dict(name="norm_step_b128", op="norm", **MFA, rows=128, rotary=256, axes=3, pairing="half", type="bf16"),
        # a prompt of text and images
        dict(name="norm_prompt", op="norm", **MFA, rows=8191, rotary=256, axes=3, pairing="half", type="bf16"),
        # the gradient of a training batch
        dict(name="grad_batch", op="grad", **MFA, rows=8191, rotary=256, axes=3, pairing="half", type="bf16"),
        # the gradient of image patches in fp32, adjacent pairs, part of each head turned
        dict(name="grad_patches_fp32", op="grad", **GQA, rows=1021, rotary=96, axes=2, pairing="adjacent", type="fp32"),
        # one sequence of a chat: latency counts
        dict(name="window_b1_l512", op="window", **MFA, batch=1, shortest=512, longest=512, tokens=1, block=64, window=128, sinks=4),
        # a batch of long contexts
        dict(name="window_b128_l8192", op="window", **MFA, batch=128, shortest=8192, longest=8192, tokens=1, block=64,
             window=4096, sinks=4),
        # grouped heads, a short window, contexts of up to 128K tokens
        dict(name="window_gqa_b32_long", op="window", **GQA, batch=32, shortest=16384, longest=131072, tokens=1, block=32,
             window=1024, sinks=16),
        # ragged lengths, two new tokens a sequence (speculative decoding), finer scales
        dict(name="window_ragged_t2", op="window", **MFA, batch=61, shortest=1, longest=8192, tokens=2, block=16, window=2047,
             sinks=67),
        # one chat, a small tree: latency counts
        dict(name="tree_b1_l2048_t8", op="tree", **MFA, batch=1, shortest=2048, longest=2048, tokens=8, block=64),
        # a usual batch of drafts
        dict(name="tree_b8_l4096_t32", op="tree", **MFA, batch=8, shortest=4096, longest=4096, tokens=32, block=64),
        # grouped heads: each tree's rows of a key head fit few tiles, the cache's bytes count
        dict(name="tree_gqa_b48_l4096_t8", op="tree", **GQA, batch=48, shortest=4096, longest=4096, tokens=8, block=32),
        # ragged lengths, the largest trees
        dict(name="tree_ragged_t61", op="tree", **MFA, batch=7, shortest=61, longest=8192, tokens=61, block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "grad", "window", "window", "tree", "tree"])
    shape = rng.choice([MFA, GQA, dict(heads=32, kv_heads=8, width=128), dict(heads=40, kv_heads=8, width=128),
                        dict(heads=24, kv_heads=2, width=256)])
    row = shape["kv_heads"] * shape["width"]
    if op in ("norm", "grad"):
        axes, kind = rng.choice([1, 2, 3, 4]), rng.choice(["bf16", "bf16", "fp32"])
        rotary = rng.choice([shape["width"], 2 * rng.randint(axes, shape["width"] // 2)])
        return dict(op=op, **shape, rows=_log(rng, 1, 8191 if kind == "bf16" else 4095), rotary=rotary, axes=axes,
                    pairing=rng.choice(["half", "adjacent"]), type=kind)
    longest = _log(rng, 1, 131072)
    if op == "window":
        tokens, window, sinks = rng.choice([1, 1, 2, 3, 4]), _log(rng, 1, 8192), rng.choice([0, _log(rng, 1, 256)])
        seen = min(longest, window + sinks)
        batch = max(1, min(_log(rng, 1, 160), (100 << 20) // (seen * row * tokens), (600 << 20) // (longest * row)))
        return dict(op=op, **shape, batch=batch, shortest=rng.choice([longest, 0, rng.randint(0, longest)]), longest=longest,
                    tokens=tokens, block=rng.choice([16, 32, 64]), window=window, sinks=sinks)
    tokens = _log(rng, 1, 64)
    pairs = tokens * shape["heads"] * longest
    batch = max(1, min(_log(rng, 1, 64), (100 << 20) // (longest * row), (60 << 20) // pairs))
    tokens = max(1, min(tokens, (100 << 20) // (shape["heads"] * longest)))
    return dict(op=op, **shape, batch=batch, shortest=rng.choice([longest, 0, rng.randint(0, longest)]), longest=longest,
                tokens=tokens, block=rng.choice([16, 32, 64]))


# ---------------------------------------------------------------------------- inputs

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _lengths(lo, hi, n, gen, dev):
    """n lengths in [lo, hi], the last of them hi."""
    x = torch.randint(lo, hi + 1, (n,), generator=gen, device=dev, dtype=torch.int32)
    x[-1] = hi
    return x


def _table(columns, batch, gen, dev):
    """A block table whose pages are spread over the pool, and the pool's pages (some unused)."""
    pages = batch * columns + 3
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int32)
    return order[:batch * columns].reshape(batch, columns).contiguous(), pages


def _quantised(pages, kv_heads, width, block, gen, dev):
    """Codes and scales of N(0, 1) rows, each (block, head) under its own magnitude and power-of-two scale."""
    codes = torch.empty((pages, kv_heads, PAGE, width), dtype=torch.uint8, device=dev)
    scales = torch.empty((pages, kv_heads, PAGE // block), device=dev)
    for p in range(0, pages, 4096):   # in parts: the fp32 values of a whole pool are four times its codes
        n = min(4096, pages - p)
        x = torch.randn((n, kv_heads, PAGE // block, block, width), generator=gen, device=dev)
        x *= torch.exp2(torch.rand((n, kv_heads, PAGE // block, 1, 1), generator=gen, device=dev) * 2 - 1)
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((3, 4)) / E4M3_MAX)))
        codes[p:p + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, kv_heads, PAGE, width)
        scales[p:p + n] = s
    return codes, scales


def _sections(rotary, axes):
    """The rotary pairs of each axis: as equal as they come, the first axis taking what is left."""
    pairs = rotary // 2
    rest = [pairs // axes] * (axes - 1)
    return [pairs - sum(rest)] + rest


def _trees(batch, tokens, gen, dev):
    """Ancestor masks int64 [batch, tokens]: node i hangs from one of the nodes before it, or from the cache's
    last token; bit j of node i's mask is set where j is i or one of its ancestors."""
    masks = torch.zeros((batch, tokens), dtype=torch.int64, device=dev)
    for i in range(tokens):
        parent = torch.randint(-1, i, (batch, 1), generator=gen, device=dev) if i else torch.full((batch, 1), -1, device=dev)
        above = torch.where(parent >= 0, masks.gather(1, parent.clamp(min=0)), 0)
        masks[:, i:i + 1] = above | (1 << i if i < 63 else -1 << 63)
    return masks


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    H, G, d = case["heads"], case["kv_heads"], case["width"]
    st = dict(case=case)
    if case["op"] in ("norm", "grad"):
        N, dt = case["rows"], torch.bfloat16 if case["type"] == "bf16" else torch.float32
        for name, n in (("q", H), ("k", G)):   # heads of different magnitudes, as projections give them
            size = torch.exp2(torch.rand((1, n, 1), generator=gen, device=dev) * 4 - 2)
            st[name] = (torch.randn((N, n, d), generator=gen, device=dev) * size).to(dt)
            st["w" + name] = (1 + 0.25 * torch.randn((d,), generator=gen, device=dev)).to(dt)
            if case["op"] == "grad":
                st["d" + name] = torch.randn((N, n, d), generator=gen, device=dev).to(dt)
        far = torch.randint(0, 1 << 17, (1, 1), generator=gen, device=dev)
        near = torch.randint(0, 1024, (case["axes"], N), generator=gen, device=dev)
        near[0] += far[0] + torch.arange(N, device=dev)   # the first axis walks on, as time and text positions do
        st["positions"] = near.to(torch.int32).contiguous()
        st["sections"] = _sections(case["rotary"], case["axes"])
        if own:
            import decode_attention_02_gb300 as mfa
            st["norm"] = mfa.NormRope(d, st["sections"], eps=EPS, theta=1e4, pairing=case["pairing"], device=dev)
        return st
    B, block, T = case["batch"], case["block"], case["tokens"]
    lens = _lengths(case["shortest"], case["longest"], B, gen, dev)
    columns = max(1, -(-case["longest"] // PAGE))
    st["q"] = torch.randn((B * T, H, d), generator=gen, device=dev).bfloat16()
    st["lens"] = lens
    st["table"], pages = _table(columns, B, gen, dev)
    for name in ("k", "v"):
        st[name + "_codes"], st[name + "_scale"] = _quantised(pages, G, d, block, gen, dev)
    if case["op"] == "tree":
        st["tree"] = _trees(B, T, gen, dev)
    if own:
        import decode_attention_02_gb300 as mfa
        shape = dict(num_q_heads=H, num_kv_heads=G, head_dim=d, scale_tokens=block, host_seq_lens=lens.tolist(), device=dev)
        if case["op"] == "window":
            st["cache"] = mfa.BlockDecoder(B, columns, pages, tokens_per_seq=T, window=case["window"], sinks=case["sinks"], **shape)
        else:
            st["cache"] = mfa.TreeDecoder(B, columns, pages, tree_tokens=T, **shape)
    return st


# ---------------------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if op == "norm":
        if own:
            return st["norm"](st["q"], st["k"], st["wq"], st["wk"], st["positions"])
        return _norm(st)
    if op == "grad":
        if own:
            return st["norm"].grad(st["dq"], st["dk"], st["q"], st["k"], st["wq"], st["wk"], st["positions"])
        return _grad(st)
    cache = (st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
    if op == "window":
        if own:
            return st["cache"](st["q"], *cache)
        return _window(st)
    if own:
        return st["cache"](st["q"], *cache, st["tree"])
    return _tree(st)


def _angles(st):
    """cos and sin [rows, 1, pairs] of position times frequency, the angles in 64 bits."""
    case, dev, r = st["case"], st["q"].device, st["case"]["rotary"]
    i = torch.arange(r // 2, device=dev, dtype=torch.float64)
    axis = torch.repeat_interleave(torch.arange(len(st["sections"])), torch.tensor(st["sections"])).to(dev)
    angle = st["positions"].double()[axis].T * torch.pow(1e4, -2 * i / r)
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _turn(case, x, cos, sin):
    """x'(first) = x(first) cos - x(second) sin, x'(second) = x(second) cos + x(first) sin for each pair."""
    r, half = case["rotary"], case["pairing"] == "half"
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if half else (x[..., 0:r:2], x[..., 1:r:2])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([ya, yb], -1) if half else torch.stack([ya, yb], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _norm(st):
    """y = turn(x r w), r = (mean x^2 + eps)^(-1/2) over each head."""
    cos, sin = _angles(st)
    outs = []
    for name in ("q", "k"):
        x = st[name].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        outs.append(_turn(st["case"], x * r * st["w" + name].float(), cos, sin).to(st[name].dtype))
    return outs


def _grad(st):
    """With g = turn back(dy), h = x r: dx = r (g w - h mean(g w h)), dw = sum over rows and heads of g h."""
    cos, sin = _angles(st)
    grads, weights = [], []
    for name in ("q", "k"):
        x = st[name].float()
        g = _turn(st["case"], st["d" + name].float(), cos, -sin)
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        h = x * r
        u = g * st["w" + name].float()
        grads.append((r * (u - h * (u * h).mean(-1, keepdim=True))).to(st[name].dtype))
        weights.append((g * h).sum((0, 1), dtype=torch.float64).float())
    return grads + weights


def _values(st, name, at, held):
    """[B, G, n, d] values of the tokens at [B, n], zeros where they are not held."""
    case, table = st["case"], st["table"].long()
    at = torch.where(held, at, 0)
    page, slot = table.gather(1, at // PAGE), at % PAGE
    x = st[name + "_codes"][page, :, slot].view(torch.float8_e4m3fn).float()                 # [B, n, G, d]
    x = x * st[name + "_scale"][page, :, slot // case["block"]][..., None]
    return torch.where(held[..., None, None], x, 0.0).transpose(1, 2)


def _attend(st, at, held, seen):
    """Softmax attention of q over the tokens at [B, n]; seen [B, T, n]."""
    case = st["case"]
    H, G, d, T = case["heads"], case["kv_heads"], case["width"], case["tokens"]
    B, n = at.shape
    qf = st["q"].float().view(B, T, G, H // G, d).permute(0, 2, 1, 3, 4).reshape(B, G, T * (H // G), d)
    s = (qf @ _values(st, "k", at, held).transpose(2, 3) * d ** -0.5).view(B, G, T, H // G, n)
    s = torch.where(seen[:, None, :, None], s, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = (e.view(B, G, T * (H // G), n) @ _values(st, "v", at, held)).view(B, G, T, H // G, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total)).squeeze(-1)
    out = o.permute(0, 2, 1, 3, 4).reshape(B * T, H, d).bfloat16()
    return [out, lse.permute(0, 2, 1, 3).reshape(B * T, H)]


def _window(st):
    """Token i of the T new ones, at position p = L - T + i, sees t <= p with t < sinks or t > p - window."""
    case, lens = st["case"], st["lens"].long()
    T, W, S = case["tokens"], case["window"], case["sinks"]
    dev = lens.device
    n = min(W + T - 1, case["longest"])
    last = lens[:, None] - n + torch.arange(n, device=dev)
    first = torch.arange(S, device=dev).expand(lens.shape[0], S)
    at = torch.cat([first, last], 1)
    held = torch.cat([first < lens[:, None], last >= S], 1)
    p = (lens[:, None] - T + torch.arange(T, device=dev))[..., None]
    t = at[:, None]
    seen = held[:, None] & (t <= p) & ((t < S) | (t > p - W))
    return _attend(st, at, held, seen)


def _tree(st):
    """Node i sees the tokens before the tree's T, and those of the tree that its mask names."""
    case, lens = st["case"], st["lens"].long()
    T = case["tokens"]
    at = torch.arange(case["longest"], device=lens.device).expand(lens.shape[0], -1)
    held = at < lens[:, None]
    node = at - (lens[:, None] - T)                                                          # < 0 before the tree
    bit = (st["tree"][..., None] >> node.clamp(0, 63)[:, None]) & 1
    seen = held[:, None] & ((node[:, None] < 0) | (bit == 1))
    return _attend(st, at, held, seen)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    H, G, d = case["heads"], case["kv_heads"], case["width"]
    if case["op"] in ("norm", "grad"):
        N, r, size = case["rows"], case["rotary"], 2 if case["type"] == "bf16" else 4
        n = N * (H + G) * d
        if case["op"] == "norm":   # rows in and out, positions, weights; squares, products, the turn
            return dict(bytes=n * size * 2 + 4 * case["axes"] * N + 2 * d * size, flops=n * 4 + N * (H + G) * r * 3)
        # the rows, their gradients in and out; weights and their gradients
        return dict(bytes=n * size * 3 + 4 * case["axes"] * N + 2 * d * (size + 4), flops=n * 12 + N * (H + G) * r * 3)
    B, T, block = case["batch"], case["tokens"], case["block"]
    mean = (case["shortest"] + case["longest"]) / 2 if B > 1 else case["longest"]
    if case["op"] == "window":
        mean = min(mean, case["window"] + case["sinks"])
    row = 2 * G * d                                                             # bytes of a token's codes, K and V
    scales = 2 * G * 4 / block
    rest = B * T * H * (d * 2 * 2 + 4) + 4 * B + (8 * B * T if case["op"] == "tree" else 0)
    return dict(bytes=mean * B * (row + scales + 4 / PAGE) + rest, flops=4.0 * mean * B * T * H * d)


# ---------------------------------------------------------------------------- in 64 bits, from the definition

def _exact_norm(case, st):
    dev, r, d = st["q"].device, case["rotary"], case["width"]
    pos = st["positions"].cpu().double()
    axis_of = [a for a, n in enumerate(st["sections"]) for _ in range(n)]
    unit = []
    for i in range(r // 2):
        w = (pos[axis_of[i]] * 10000.0 ** (-2.0 * i / r)).to(dev)[:, None]
        first, second = (i, i + r // 2) if case["pairing"] == "half" else (2 * i, 2 * i + 1)
        unit.append((first, second, torch.polar(torch.ones_like(w), w)))
    outs, weights = [], []
    for name in ("q", "k"):
        x, w = st[name].double(), st["w" + name].double()
        r = 1 / torch.sqrt(x.square().sum(-1) / d + EPS)
        if case["op"] == "norm":
            y = torch.einsum("nhd,nh,d->nhd", x, r, w)
            for first, second, e in unit:
                z = torch.complex(y[..., first], y[..., second]) * e
                y[..., first], y[..., second] = z.real, z.imag
            outs.append(y)
            continue
        g = st["d" + name].double()
        for first, second, e in unit:
            z = torch.complex(g[..., first], g[..., second]) * e.conj()
            g[..., first], g[..., second] = z.real, z.imag
        # y = x r(x): dx_i = r g_i w_i - r^3 x_i / d * sum_j g_j w_j x_j
        dot = torch.einsum("nhd,d,nhd->nh", g, w, x)
        outs.append(torch.einsum("nhd,nh,d->nhd", g, r, w) - torch.einsum("nhd,nh->nhd", x, dot * r ** 3 / d))
        weights.append(torch.einsum("nhd,nhd,nh->d", g, x, r))
    return outs + weights


def exact(case, seed):
    """Sequence by sequence in fp64, from the inputs of prepare()."""
    st = prepare(case, seed)
    if case["op"] in ("norm", "grad"):
        return _exact_norm(case, st)
    H, G, d, block, T = case["heads"], case["kv_heads"], case["width"], case["block"], case["tokens"]
    dev = _device()
    table, lens = st["table"].cpu().tolist(), st["lens"].tolist()
    out = torch.zeros((case["batch"] * T, H, d), dtype=torch.float64, device=dev)
    lse = torch.full((case["batch"] * T, H), float("-inf"), dtype=torch.float64, device=dev)
    masks = st["tree"].cpu().tolist() if case["op"] == "tree" else None
    for b, L in enumerate(lens):
        if L == 0:
            continue
        # the pages that hold a token which anyone sees
        pages = list(range(-(-L // PAGE)))
        if case["op"] == "window":
            low = max(0, L - T - case["window"] + 1)
            pages = [j for j in pages if j * PAGE < case["sinks"] or (j + 1) * PAGE > low]
        t = (torch.tensor(pages)[:, None] * PAGE + torch.arange(PAGE)).flatten().to(dev)
        idx = torch.tensor([table[b][j] for j in pages], device=dev)
        rows = []
        for name in ("k", "v"):
            x = st[name + "_codes"][idx].view(torch.float8_e4m3fn).double()     # [P, G, 64, d]
            x = x * st[name + "_scale"][idx].double().repeat_interleave(block, 2)[..., None]
            rows.append(x.transpose(0, 1).reshape(G, -1, d))
        for i in range(T):
            p = L - T + i
            if case["op"] == "window":
                see = (t <= p) & ((t < case["sinks"]) | (t > p - case["window"]))
            else:
                named = torch.zeros(T + 1, dtype=torch.bool)
                for j in range(T):
                    named[j] = bool(masks[b][i] >> j & 1)
                node = t - (L - T)
                see = (t < L) & ((node < 0) | named.to(dev)[node.clamp(0, T)])
            if not bool(see.any()):
                continue
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                logit = st["q"][b * T + i, hs].double() @ rows[0][g][see].T / math.sqrt(d)
                lse[b * T + i, hs] = torch.logsumexp(logit, -1)
                out[b * T + i, hs] = torch.softmax(logit, -1) @ rows[1][g][see]
    return [out, lse]
