"""The serving-step operators around the block-scaled 8-bit KV cache, as measured cases.

Three operators, in the order in which a decode step uses them:

``rope``    rotary positions with several axes (time, height, width) of the query heads and
            of the new key rows;
``append``  the new key and value rows into a paged cache of e4m3 codes with one fp32 scale
            for each block of tokens and key/value head;
``decode``  attention of 1 to 4 new tokens a sequence over that cache.

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
MFA = dict(heads=64, kv_heads=1, width=256)     # one shared key head and one shared value head
GQA = dict(heads=64, kv_heads=4, width=128)     # grouped heads


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence of a short chat: latency counts
        dict(name="decode_b1_l512", op="decode", **MFA, batch=1, shortest=512, longest=512, tokens=1, block=64),
        # a usual serving batch at a 4K context
        dict(name="decode_b32_l4096", op="decode", **MFA, batch=32, shortest=4096, longest=4096, tokens=1, block=64),
        # a full batch at a 4K context
        dict(name="decode_b128_l4096", op="decode", **MFA, batch=128, shortest=4096, longest=4096, tokens=1, block=64),
        # a few very long contexts, split over the whole card
        dict(name="decode_b4_long", op="decode", **MFA, batch=4, shortest=16384, longest=131072, tokens=1, block=64),
        # ragged lengths, two new tokens a sequence (speculative decoding), finer scales
        dict(name="decode_ragged_t2", op="decode", **MFA, batch=61, shortest=1, longest=8192, tokens=2, block=16),
        # grouped heads at the same context
        dict(name="decode_gqa_b32_l4096", op="decode", **GQA, batch=32, shortest=4096, longest=4096, tokens=1, block=32),
        # the new rows of one decode step
        dict(name="append_step_b128", op="append", **MFA, batch=128, shortest=1, longest=1, held=4095, block=64),
        # whole prompts of odd lengths into an empty cache
        dict(name="append_prompt", op="append", **MFA, batch=24, shortest=700, longest=8191, held=0, block=64),
        # a prompt's next chunk behind what is held, grouped heads
        dict(name="append_chunk_gqa", op="append", **GQA, batch=7, shortest=1000, longest=2049, held=3001, block=16),
        # the query heads and the new key of one decode step
        dict(name="rope_step_b128", op="rope", **MFA, rows=128, rotary=256, axes=3, pairing="half"),
        # a prompt of text and images
        dict(name="rope_prompt", op="rope", **MFA, rows=8191, rotary=256, axes=3, pairing="half"),
        # height and width of image patches, adjacent pairs, part of each head
        dict(name="rope_patches_gqa", op="rope", **GQA, rows=4097, rotary=96, axes=2, pairing="adjacent"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "rope"])
    shape = rng.choice([MFA, GQA, dict(heads=32, kv_heads=8, width=128), dict(heads=40, kv_heads=8, width=128),
                        dict(heads=24, kv_heads=2, width=256)])
    row = shape["kv_heads"] * shape["width"]
    if op == "decode":
        longest, tokens = _log(rng, 1, 131072), rng.choice([1, 1, 2, 3, 4])
        batch = max(1, min(_log(rng, 1, 160), (100 << 20) // (longest * row * tokens)))
        shortest = rng.choice([longest, 0, rng.randint(0, longest)])
        return dict(op=op, **shape, batch=batch, shortest=shortest, longest=longest, tokens=tokens,
                    block=rng.choice([16, 32, 64]))
    if op == "append":
        longest = rng.choice([1, rng.randint(1, 4), _log(rng, 1, 8192)])
        batch = max(1, min(_log(rng, 1, 160), (24 * 8191 * 256) // (longest * row)))
        return dict(op=op, **shape, batch=batch, shortest=rng.choice([longest, rng.randint(0, longest)]), longest=longest,
                    held=rng.choice([0, rng.randint(0, 4096)]), block=rng.choice([16, 32, 64]))
    axes = rng.choice([1, 2, 3, 4])
    rotary = rng.choice([shape["width"], 2 * rng.randint(axes, shape["width"] // 2)])
    return dict(op=op, **shape, rows=_log(rng, 1, 8191), rotary=rotary, axes=axes, pairing=rng.choice(["half", "adjacent"]))


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
    for p in range(0, pages, 1024):   # in parts: the fp32 values of a whole pool are four times its codes
        n = min(1024, pages - p)
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


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    H, G, d = case["heads"], case["kv_heads"], case["width"]
    st = dict(case=case)
    if case["op"] == "rope":
        N = case["rows"]
        st["q"] = torch.randn((N, H, d), generator=gen, device=dev).bfloat16()
        st["k"] = torch.randn((N, G, d), generator=gen, device=dev).bfloat16()
        far = torch.randint(0, 1 << 17, (1, 1), generator=gen, device=dev)
        near = torch.randint(0, 1024, (case["axes"], N), generator=gen, device=dev)
        near[0] += far[0] + torch.arange(N, device=dev)   # the first axis walks on, as time and text positions do
        st["positions"] = near.to(torch.int32).contiguous()
        st["sections"] = _sections(case["rotary"], case["axes"])
        if own:
            import decode_attention_02_gb300 as mfa
            st["rope"] = mfa.Rope(d, st["sections"], theta=1e4, pairing=case["pairing"], device=dev)
        return st
    B, block = case["batch"], case["block"]
    if case["op"] == "decode":
        T = case["tokens"]
        lens = _lengths(case["shortest"], case["longest"], B, gen, dev)
        columns = max(1, -(-case["longest"] // PAGE))
        st["q"] = torch.randn((B * T, H, d), generator=gen, device=dev).bfloat16()
        st["lens"] = lens
    else:
        new = _lengths(case["shortest"], case["longest"], B, gen, dev)
        held = torch.full((B,), case["held"], dtype=torch.int32, device=dev)
        if case["held"]:
            held -= torch.randint(0, min(PAGE, case["held"] + 1), (B,), generator=gen, device=dev, dtype=torch.int32)
        columns = max(1, -(-(case["held"] + case["longest"]) // PAGE))
        st["offsets"] = torch.cat([new.new_zeros(1), new.cumsum(0, dtype=torch.int32)])
        st["held"] = held
        st["rows"] = int(st["offsets"][-1])
        for name in ("k_new", "v_new"):
            x = torch.randn((st["rows"], G, d), generator=gen, device=dev)
            st[name] = (x * torch.exp2(torch.rand((st["rows"], G, 1), generator=gen, device=dev) * 4 - 2)).bfloat16()
    st["table"], pages = _table(columns, B, gen, dev)
    for name in ("k", "v"):
        st[name + "_codes"], st[name + "_scale"] = _quantised(pages, G, d, block, gen, dev)
    if own:
        import decode_attention_02_gb300 as mfa
        host = st["lens"].tolist() if case["op"] == "decode" else None
        st["cache"] = mfa.BlockDecoder(B, columns, pages, num_q_heads=H, num_kv_heads=G, head_dim=d, scale_tokens=block,
                                       tokens_per_seq=case.get("tokens", 1), host_seq_lens=host, device=dev)
    return st


# ---------------------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if op == "rope":
        if own:
            return st["rope"](st["q"], st["k"], st["positions"])
        return _rope(st)
    if op == "append":
        if own:
            st["cache"].append(st["k_new"], st["v_new"], st["held"], st["table"], st["k_codes"], st["v_codes"],
                               st["k_scale"], st["v_scale"], offsets=st["offsets"], max_new=st["case"]["longest"])
        else:
            for x, codes, scale in ((st["k_new"], st["k_codes"], st["k_scale"]), (st["v_new"], st["v_codes"], st["v_scale"])):
                _append(st, x, codes, scale)
        return [st["k_codes"].view(torch.float8_e4m3fn), st["k_scale"], st["v_codes"].view(torch.float8_e4m3fn),
                st["v_scale"]]
    if own:
        return st["cache"](st["q"], st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
    return _decode(st)


def _pair_axes(sections):
    return torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))


def _rope(st):
    """x'(first) = x(first) cos - x(second) sin, x'(second) = x(second) cos + x(first) sin for each pair."""
    case = st["case"]
    dev, r = st["q"].device, case["rotary"]
    i = torch.arange(r // 2, device=dev, dtype=torch.float64)
    angle = st["positions"].double()[_pair_axes(st["sections"]).to(dev)].T * torch.pow(1e4, -2 * i / r)
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = case["pairing"] == "half"
    outs = []
    for x in (st["q"], st["k"]):
        x = x.float()
        a, b = (x[..., :r // 2], x[..., r // 2:r]) if half else (x[..., 0:r:2], x[..., 1:r:2])
        ya, yb = a * cos - b * sin, b * cos + a * sin
        y = torch.cat([ya, yb], -1) if half else torch.stack([ya, yb], -1).flatten(-2)
        outs.append(torch.cat([y, x[..., r:]], -1).bfloat16())
    return outs


def _append(st, new, codes, scale):
    """Each touched block takes the smallest power-of-two scale that holds its new rows, or keeps its
    own where that is larger; rows that it held are coded again where its scale rises."""
    case = st["case"]
    block, G, d = case["block"], case["kv_heads"], case["width"]
    dev = new.device
    held, offs = st["held"].long(), st["offsets"].long()
    count = offs[1:] - offs[:-1]
    first = held // block
    most = (case["longest"] + block - 2) // block + 1
    idx = first[:, None] + torch.arange(most, device=dev)                       # [B, M] blocks of the sequence
    live = (idx * block < (held + count)[:, None]) & (count > 0)[:, None]
    b, m = live.nonzero(as_tuple=True)
    blk = idx[b, m]
    page, sub = st["table"].long()[b, blk * block // PAGE], blk % (PAGE // block)
    pos = blk[:, None] * block + torch.arange(block, device=dev)                # [touched, block] positions
    is_old = pos < held[b][:, None]
    is_new = ~is_old & (pos < (held + count)[b][:, None])
    row = (offs[b][:, None] + pos - held[b][:, None]).clamp(0, new.shape[0] - 1)
    x = torch.where(is_new[..., None, None], new[row].float(), 0.0)             # [touched, block, G, d]
    a = x.abs().amax((1, 3))
    part, e = torch.frexp(a.double() / E4M3_MAX)                                # in [0.5, 1) * 2^e; 0 gives 0
    e = torch.where(part == 0.5, e - 1, e)
    need = torch.ldexp(torch.ones_like(a), torch.where(a > 0, e, -126).clamp(min=-126))
    old_s = scale[page, :, sub]
    s = torch.where(is_old.any(1)[:, None], torch.maximum(old_s, need), need)
    view = codes.view(codes.shape[0], G, PAGE // block, block, d)
    old_c = view[page, :, sub]                                                  # [touched, G, block, d]
    ratio = (old_s / s)[..., None, None]
    kept = (old_c.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
    fresh = (x.permute(0, 2, 1, 3) / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.where(is_new[:, None, :, None], fresh, torch.where((is_old[:, None, :, None]) & (ratio < 1), kept, old_c))
    view[page, :, sub] = out
    scale[page, :, sub] = s


def _decode(st):
    case = st["case"]
    H, G, d, T, block = case["heads"], case["kv_heads"], case["width"], case["tokens"], case["block"]
    q, lens, table = st["q"], st["lens"].long(), st["table"].long()
    B = lens.shape[0]
    S = table.shape[1] * PAGE
    dev = q.device
    t = torch.arange(S, device=dev)
    held = (t < lens[:, None])[:, None, :, None]                                # tokens past the length are not read

    def values(codes, scale):
        x = codes[table].view(torch.float8_e4m3fn).float()                      # [B, P, G, 64, d]
        x = x.view(B, -1, G, PAGE // block, block, d) * scale[table][..., None, None]
        x = x.permute(0, 2, 1, 3, 4, 5).reshape(B, G, S, d)
        return torch.where(held, x, 0.0)

    seen = t < (lens[:, None] - (T - 1) + torch.arange(T, device=dev))[..., None]          # [B, T, S]
    qf = q.float().view(B, T, G, H // G, d).permute(0, 2, 1, 3, 4).reshape(B, G, T * (H // G), d)
    s = (qf @ values(st["k_codes"], st["k_scale"]).transpose(2, 3) * d ** -0.5).view(B, G, T, H // G, S)
    s = torch.where(seen[:, None, :, None], s, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = (e.view(B, G, T * (H // G), S) @ values(st["v_codes"], st["v_scale"])).view(B, G, T, H // G, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total)).squeeze(-1)
    out = o.permute(0, 2, 1, 3, 4).reshape(B * T, H, d).bfloat16()
    return [out, lse.permute(0, 2, 1, 3).reshape(B * T, H)]


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    H, G, d = case["heads"], case["kv_heads"], case["width"]
    if case["op"] == "rope":
        N, r = case["rows"], case["rotary"]
        return dict(bytes=N * (H + G) * d * 2 * 2 + 4 * case["axes"] * N, flops=N * (H + G) * r * 3)
    B, block = case["batch"], case["block"]
    mean = (case["shortest"] + case["longest"]) / 2 if B > 1 else case["longest"]
    tokens = mean * B
    row = 2 * G * d                                                             # bytes of a token's codes, K and V
    scales = 2 * G * 4 / block
    if case["op"] == "append":   # rows in, codes out; the scale of a begun block is read and written
        return dict(bytes=tokens * (2 * row + row + scales) + B * (12 + 2 * 2 * G * 4), flops=tokens * row * 2)
    T = case["tokens"]
    return dict(bytes=tokens * (row + scales + 4 / PAGE) + B * T * H * (d * 2 * 2 + 4) + 4 * B, flops=4.0 * tokens * T * H * d)


# ---------------------------------------------------------------------------- in 64 bits, from the definition

def exact(case, seed):
    """Sequence by sequence in fp64, from the inputs of prepare()."""
    st = prepare(case, seed)
    H, G, d = case["heads"], case["kv_heads"], case["width"]
    dev = _device()
    if case["op"] == "rope":
        r = case["rotary"]
        pos = st["positions"].cpu().double()
        outs = []
        axis_of = [a for a, n in enumerate(st["sections"]) for _ in range(n)]
        for x in (st["q"], st["k"]):
            y = x.double()
            for i in range(r // 2):
                w = (pos[axis_of[i]] * 10000.0 ** (-2.0 * i / r)).to(dev)[:, None]
                first, second = (i, i + r // 2) if case["pairing"] == "half" else (2 * i, 2 * i + 1)
                z = torch.complex(x[..., first].double(), x[..., second].double()) * torch.polar(torch.ones_like(w), w)
                y[..., first], y[..., second] = z.real, z.imag
            outs.append(y)
        return outs
    block = case["block"]
    table = st["table"].cpu().tolist()
    if case["op"] == "append":
        if st["rows"] > 40000:   # a host loop over blocks
            return None
        held, offs = st["held"].tolist(), st["offsets"].tolist()
        outs = []
        for name in ("k", "v"):
            new = st[name + "_new"].double().cpu()
            codes, scale = st[name + "_codes"].cpu(), st[name + "_scale"].double().cpu()
            value = codes.view(torch.float8_e4m3fn).double()
            for b in range(case["batch"]):
                n, t = offs[b + 1] - offs[b], held[b]
                end = t + n
                while t < end:   # one block at a time
                    stop = min(end, (t // block + 1) * block)
                    page, slot, begin = table[b][t // PAGE], t % PAGE, t % PAGE // block * block
                    x = new[offs[b] + t - held[b]:offs[b] + stop - held[b]]      # [rows, G, d]
                    for g in range(G):
                        a = float(x[:, g].abs().max())
                        e = -126
                        if a > 0:
                            e = math.frexp(a / E4M3_MAX)[1]
                            e = max(e - 1 if a <= E4M3_MAX * 2.0 ** (e - 1) else e, -126)
                        s = 2.0 ** e
                        if slot > begin:
                            was = float(scale[page, g, begin // block])
                            s = max(s, was)
                            if s > was:
                                old = value[page, g, begin:slot] * (was / s)
                                value[page, g, begin:slot] = old.float().to(torch.float8_e4m3fn).double()
                        scale[page, g, begin // block] = s
                        value[page, g, slot:slot + stop - t] = (x[:, g] / s).float().to(torch.float8_e4m3fn).double()
                    t = stop
            outs += [value, scale]
        return outs
    T = case["tokens"]
    lens = st["lens"].tolist()
    out = torch.zeros((case["batch"] * T, H, d), dtype=torch.float64, device=dev)
    lse = torch.full((case["batch"] * T, H), float("-inf"), dtype=torch.float64, device=dev)
    for b, L in enumerate(lens):
        if L == 0:
            continue
        pages = torch.tensor(table[b][:-(-L // PAGE)], device=dev)
        rows = []
        for name in ("k", "v"):
            x = st[name + "_codes"][pages].view(torch.float8_e4m3fn).double()   # [P, G, 64, d]
            x = x * st[name + "_scale"][pages].double().repeat_interleave(block, 2)[..., None]
            rows.append(x.transpose(0, 1).reshape(G, -1, d)[:, :L])
        for i in range(T):
            n = L - (T - 1) + i
            if n <= 0:
                continue
            for g in range(G):
                hs = slice(g * (H // G), (g + 1) * (H // G))
                logit = st["q"][b * T + i, hs].double() @ rows[0][g, :n].T / math.sqrt(d)
                lse[b * T + i, hs] = torch.logsumexp(logit, -1)
                out[b * T + i, hs] = torch.softmax(logit, -1) @ rows[1][g, :n]
    return [out, lse]
