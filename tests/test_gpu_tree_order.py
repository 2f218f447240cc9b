"""Trees over many tiles, again and again: a tile's scores lie where the weights of the tile before last lay, and must not go
there before the product that reads those is complete."""
import pytest
import torch

import seen_reference as seen
import test_gpu_tree as trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape, lens, tokens", [
    (trees.MFA, [4096, 3001], 32), (trees.MFA, [2500], 2), (trees.GQA, [2200, 777, 1500], 8), (trees.SINGLE, [4096], 61)])
def test_many_tiles_give_the_same_bits_every_time(shape, lens, tokens):
    c = trees.case(lens, tokens, **shape, scale_tokens=16, seed=tokens)
    dec = trees.decoder(c, force_ctas=2, **trees.CHECK)   # few CTAs: long runs of tiles
    args = trees.device(c)
    out, lse = dec(*args)
    seen.check(out, lse, trees.expect(c))
    for _ in range(40):
        again, again_lse = dec(*args)
        assert torch.equal(again, out) and torch.equal(again_lse, lse)
