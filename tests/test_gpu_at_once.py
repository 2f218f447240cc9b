"""Calls on two streams at once, and replayed graphs that share a device, on the GPU: trees, windows, normed rotary rows."""
import pytest
import torch

import decode_attention_02_gb300 as mfa
import test_gpu_tree as trees
import test_gpu_window as windows
from test_gpu_block import DEV

pytestmark = pytest.mark.gpu


def makers():
    """(name, a function that makes a call with what it owns): the calls of one kind have different inputs."""
    def tree(seed, **kw):
        c = trees.case([900 + 300 * seed, 30, 2500], 9, **trees.GQA, seed=seed, scale_tokens=32)
        d, dec = trees.device(c), trees.decoder(c, **kw)
        return lambda: dec(*d)

    def window(seed, **kw):
        c = windows.case([3000 + 500 * seed, 70, 1], 700, 5, poison=False, **windows.MFA, scale_tokens=64, seed=seed)
        d, dec = windows.device(c), windows.decoder(c, 700, 5, **kw)
        return lambda: dec(*d)

    norm = mfa.NormRope(128, [40, 24])

    def grad(seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        x = [torch.randn((700, h, 128), generator=gen, device=DEV, dtype=torch.bfloat16) for h in (24, 4, 24, 4)]
        w = [torch.rand(128, generator=gen, device=DEV) for _ in range(2)]
        pos = torch.randint(0, 10 ** 5, (2, 700), generator=gen, device=DEV, dtype=torch.int32)
        return lambda: norm.grad(*x, *w, pos)

    return [("tree", tree), ("tree in parts", lambda seed: tree(seed, force_ctas=13)), ("window", window),
            ("window in parts", lambda seed: window(seed, force_ctas=7)), ("gradient", grad)]


@pytest.mark.parametrize("name", ["tree", "tree in parts", "window", "window in parts", "gradient"])
def test_two_calls_at_once(name):
    make = dict(makers())[name]
    calls = [make(1), make(2)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(8):
        for i, (call, stream) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(stream):
                got[i].append(call())
    torch.cuda.synchronize()
    for results, right in zip(got, want):
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, right))


@pytest.mark.parametrize("name", ["tree in parts", "window in parts", "gradient"])
def test_two_graphs_of_one_object(name):
    """Captured one after the other, replayed in turn: what they share holds no state from one to the next."""
    call = dict(makers())[name](1)
    want = call()
    torch.cuda.synchronize()
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(call())
        graphs.append(g)
    for _ in range(3):
        for g, r in zip(graphs, results):
            for x in r:
                x.fill_(7)
            g.replay()
        torch.cuda.synchronize()
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
