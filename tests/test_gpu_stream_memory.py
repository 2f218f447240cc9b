"""Memory that a call on a given stream makes anew, and a tree decoder's own buffers, on the GPU."""
import pytest
import torch

import decode_attention_02_gb300 as mfa
from test_gpu_block import DEV
from test_gpu_streams import busy, given_out_again
from test_gpu_tree import GQA, case, decoder, device

pytestmark = pytest.mark.gpu


def calls():
    """Calls on a stream: name, what it takes (made at once), and its results."""
    c = case([900, 30], 5, **GQA, seed=3)
    d, dec = device(c), decoder(c)
    q, k = (torch.randn(301, h, 128, device=DEV, dtype=torch.bfloat16) for h in (8, 2))
    w = torch.ones(128, device=DEV)
    pos = torch.arange(301, dtype=torch.int32, device=DEV)[None]
    rope, norm = mfa.Rope(128, [64]), mfa.NormRope(128, [64])
    torch.cuda.synchronize()
    yield "tree", lambda s: dec(*d, stream=s)
    yield "rope", lambda s: rope(q, k, pos, stream=s)
    yield "norm", lambda s: norm(q, k, w, w, pos, stream=s)
    yield "grad", lambda s: norm.grad(q, k, q, k, w, w, pos, stream=s)


@pytest.mark.parametrize("handle", [False, True])
def test_results_are_not_made_where_the_current_stream_still_writes(handle):
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    for name, call in calls():
        want = call(stream)
        torch.cuda.synchronize()
        sizes = [x.numel() * x.element_size() for x in want]
        torch.cuda.empty_cache()
        for n in sizes:
            old = torch.empty(n, dtype=torch.uint8, device=DEV)
            torch.cuda._sleep(20_000_000)
            old.fill_(255)
            at = range(old.data_ptr(), old.data_ptr() + n)
            del old
            got = call(stream)
            for x in got:
                assert x.data_ptr() not in at, name
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_results_may_go_while_the_current_stream_reads_them():
    side = torch.cuda.Stream()
    for name, call in calls():
        call(side)
        torch.cuda.synchronize()
        got = call(side)
        torch.cuda.synchronize()
        at, n = got[0].data_ptr(), got[0].numel() * got[0].element_size()
        torch.cuda._sleep(100_000_000)
        del got
        with torch.cuda.stream(side):
            new = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(3)]
        assert at not in [x.data_ptr() for x in new] and not torch.cuda.current_stream().query(), name
        torch.cuda.synchronize()


def test_a_tree_decoder_may_go_while_the_current_stream_of_its_append_is_at_work():
    c = case([900, 30], 5, **GQA, seed=3)
    d, dec, side = device(c), decoder(c), torch.cuda.Stream()
    new = torch.ones((10, 4, 128), dtype=torch.bfloat16, device=DEV)
    positions = torch.full((2,), -1, dtype=torch.int32, device=DEV)
    dec.append(new, new, positions, d[5], *d[1:5])
    busy(side)
    with torch.cuda.stream(side):
        dec.append(new, new, positions, d[5], *d[1:5])
    at, n = dec._offsets.data_ptr(), 12
    del dec
    assert not given_out_again(at, n, side)
    torch.cuda.synchronize()
