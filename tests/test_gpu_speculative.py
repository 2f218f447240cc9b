"""The cache's operators together on the GPU, as speculative decoding of a model with normed queries and keys uses them:
prompts, a drafted tree, the accepted nodes, and a layer that sees a window.  Against 64-bit arithmetic on the rows that
the cache holds."""
import random
import types

import pytest
import torch

import decode_attention_02_gb300 as mfa
import norm_reference as norm
import seen_reference as seen
from test_gpu_tree import draft

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


@pytest.mark.parametrize("heads, kv_heads, dim, block, T", [(64, 1, 256, 64, 6), (64, 4, 128, 16, 17), (40, 8, 128, 32, 5)])
def test_prompt_tree_accept_and_window(heads, kv_heads, dim, block, T):
    gen = torch.Generator().manual_seed(dim + T)
    rng = random.Random(T)
    prompts, sections = [130, 1, 700, 61], (dim // 4, dim // 8, dim // 8)
    B, columns = len(prompts), 14
    pages = B * columns + 2
    table = torch.randperm(pages, generator=gen)[:B * columns].to(torch.int32).view(B, columns)
    op = mfa.NormRope(dim, sections, eps=EPS)
    wq, wk = ((1 + torch.randn((dim,), generator=gen) / 4).bfloat16() for _ in range(2))
    k_cache, v_cache = (torch.zeros((pages, kv_heads, 64, dim), dtype=torch.uint8, device=DEV) for _ in range(2))
    k_scale, v_scale = (torch.zeros((pages, kv_heads, 64 // block), device=DEV) for _ in range(2))
    cache = (k_cache, v_cache, k_scale, v_scale)
    tab = table.to(DEV)
    shape = dict(num_q_heads=heads, num_kv_heads=kv_heads, head_dim=dim, scale_tokens=block, flags=mfa.MFA_PLAN_CHECK)
    tree_dec = mfa.TreeDecoder(B, columns, pages, T, max_seq_len=columns * 64, **shape)
    one_dec = mfa.BlockDecoder(B, columns, pages, window=90, sinks=4, **shape)

    def rows(n):
        q, k, v = (torch.randn((n, h, dim), generator=gen).bfloat16() for h in (heads, kv_heads, kv_heads))
        return q, k, v

    def turned(q, k, positions):
        """Normed and turned rows, in place in the columns of one projection, checked against the definition."""
        n = positions.numel()
        proj = torch.cat([x.reshape(n, -1) for x in (q, k)], 1).to(DEV)
        qd, kd = proj[:, :heads * dim].view(n, heads, dim), proj[:, heads * dim:].view(n, kv_heads, dim)
        pos = positions.to(torch.int32).expand(3, n).contiguous()
        op(qd, kd, wq.to(DEV), wk.to(DEV), pos.to(DEV), q_out=qd, k_out=kd)
        for got, x, w in ((qd, q, wq), (kd, k, wk)):
            want, tol = norm.forward(x, w, pos, sections, EPS)
            assert bool(((got.cpu().double() - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8).all())
        return qd.contiguous(), kd.contiguous()

    def check(out, lse, q, lens, seen_by, rows_a_seq, bound):
        c = types.SimpleNamespace(seq_lens=torch.tensor(lens), heads=heads, kv_heads=kv_heads, dim=dim, scale_tokens=block,
                                  block_table=table, q=q.cpu(), k_cache=k_cache.cpu(), v_cache=v_cache.cpu(),
                                  k_scale=k_scale.cpu(), v_scale=v_scale.cpu())
        seen.check(out, lse, seen.decode(c, seen_by, rows_a_seq, bound))

    # the prompts into the cache
    n = sum(prompts)
    offsets = torch.tensor([0, *torch.tensor(prompts).cumsum(0).tolist()], dtype=torch.int32, device=DEV)
    _, k, v = rows(n)
    _, k = turned(torch.randn((n, heads, dim), generator=gen).bfloat16(), k, torch.cat([torch.arange(L) for L in prompts]))
    tree_dec.append(k, v.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV), tab, *cache, offsets=offsets, max_new=max(prompts))
    # a tree behind each, a node's position by its depth
    masks = [draft(T, rng) for _ in range(B)]
    depth = torch.tensor([[bin(m).count("1") - 1 for m in r] for r in masks])
    held = torch.tensor(prompts, dtype=torch.int32)
    q, k, v = rows(B * T)
    q, k = turned(q, k, (held[:, None] + depth).flatten())
    v = v.to(DEV)
    tree_dec.append(k, v, held.to(DEV), tab, *cache)
    lens = [L + T for L in prompts]
    tree = torch.tensor(masks, dtype=torch.int64, device=DEV)
    out, lse = tree_dec(q, *cache, tab, torch.tensor(lens, dtype=torch.int32, device=DEV), tree)
    check(out, lse, q, lens, lambda b, L: seen.tree_seen(L, T, masks[b]), T, seen.e4m3_and_e5m2)
    # the last node's ancestors and itself are accepted: their rows once more, from the tree's first position
    path = [[j for j in range(T) if masks[b][T - 1] >> j & 1] for b in range(B)]
    pick = torch.tensor([b * T + j for b in range(B) for j in path[b]], device=DEV)
    count = torch.tensor([len(p) for p in path])
    offsets = torch.tensor([0, *count.cumsum(0).tolist()], dtype=torch.int32, device=DEV)
    tree_dec.append(k[pick].contiguous(), v[pick].contiguous(), held.to(DEV), tab, *cache, offsets=offsets, max_new=int(count.max()))
    # the next token, whose layer sees a window and the first tokens
    held = held + count.to(torch.int32)
    q, k, v = rows(B)
    q, k = turned(q, k, held)
    one_dec.append(k, v.to(DEV), held.to(DEV), tab, *cache)
    lens = (held + 1).tolist()
    out, lse = one_dec(q, *cache, tab, torch.tensor(lens, dtype=torch.int32, device=DEV))
    check(out, lse, q, lens, lambda b, L: seen.window_seen(L, 1, 90, 4), 1, seen.two_e4m3)


def test_a_training_step_learns_its_weights():
    """A few steps of plain descent on the norms' weights run and stay finite: the gradients' own test is elsewhere."""
    gen = torch.Generator().manual_seed(2)
    op = mfa.NormRope(64, (32,), eps=EPS)
    x = torch.randn((50, 4, 64), generator=gen).to(DEV)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)[None]
    w = torch.ones(64, device=DEV)
    target, _ = op(x, None, torch.linspace(0.5, 1.5, 64, device=DEV), None, pos)
    for _ in range(3):
        y, _ = op(x, None, w, None, pos)
        dx, _, dw, _ = op.grad(y - target, None, x, None, w, None, pos)
        w = w - 0.002 * dw
        assert dx.shape == x.shape and bool(w.isfinite().all())
