"""What the block decoder and the rotary positions use on another stream stays allocated until it is done, on the GPU."""
import pytest
import torch

import block_reference as ref
import decode_attention_02_gb300 as mfa
from test_gpu_block import DEV, GQA, MFA, check, decoder, device

pytestmark = pytest.mark.gpu


def busy(side):
    """Give `side` some tens of milliseconds of work, with everything before it done."""
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)


def given_out_again(address, nbytes, side):
    """Whether memory freed at `address` is given to the current stream while `side` is still at work."""
    new = [torch.empty(nbytes, dtype=torch.uint8, device=DEV) for _ in range(3)]
    return address in [x.data_ptr() for x in new] and not side.query()   # (its memory is free once it is done)


def test_a_decoder_may_go_while_the_current_stream_of_its_last_call_is_at_work():
    c = ref.Case([900, 30], **MFA, seed=3)
    d, side = device(c), torch.cuda.Stream()
    for call in ("decode", "append"):
        dec = decoder(c, force_ctas=5)
        new = torch.ones((2, 1, 256), dtype=torch.bfloat16, device=DEV)
        positions = torch.full((2,), -1, dtype=torch.int32, device=DEV)
        dec(*d)
        busy(side)
        with torch.cuda.stream(side):
            if call == "decode":
                dec(*d)
            else:
                dec.append(new, new, positions, d[5], *d[1:5])
        at, n = dec.workspace.data_ptr(), dec.workspace.numel()
        del dec
        assert not given_out_again(at, n, side), call
        torch.cuda.synchronize()


def test_a_rope_may_go_while_the_current_stream_of_its_last_call_is_at_work():
    side = torch.cuda.Stream()
    q = torch.randn(64, 8, 128, device=DEV, dtype=torch.bfloat16)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)[None]
    rope = mfa.Rope(128, [64])
    rope(q, None, pos)
    busy(side)
    with torch.cuda.stream(side):
        rope(q, None, pos)
    at, n = rope.table.data_ptr(), rope.table.numel()
    del rope
    assert not given_out_again(at, n, side)
    torch.cuda.synchronize()


@pytest.mark.parametrize("handle", [False, True])
def test_the_inputs_of_a_call_with_a_stream_may_go(handle):
    c = ref.Case([900, 30], **GQA, seed=3)
    dec, rope, side = decoder(c), mfa.Rope(128, [64]), torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    pos = torch.arange(2, dtype=torch.int32, device=DEV)[None]

    def decode(x):
        dec(*x[:7], stream=stream)

    def append(x):
        dec.append(x[7], x[8], x[9], x[5], *x[1:5], stream=stream)

    def turn(x):
        rope(x[0], x[7], x[10], stream=stream)

    for call, used in ((decode, range(7)), (append, (1, 2, 3, 4, 5, 7, 8, 9)), (turn, (0, 7, 10))):
        for i in used:
            x = [*device(c), *(torch.ones((2, 4, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)),
                 torch.full((2,), -1, dtype=torch.int32, device=DEV), pos.clone()]
            call(x)   # (loads what is loaded at a first call)
            busy(side)
            call(x)
            at, n = x[i].data_ptr(), x[i].numel() * x[i].element_size()
            x[i] = None
            assert not given_out_again(at, n, side), (call.__name__, i)
            torch.cuda.synchronize()


def test_the_default_stream_by_its_handle():
    c = ref.Case([300, 30], **GQA, seed=5)
    d, dec = device(c), decoder(c, out_dtype=mfa.MFA_OUT_FP32)
    want = dec(*d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (0, 1):   # both name it
        with torch.cuda.stream(side):
            out, lse = dec(*d, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    check(c, out, lse)


def test_a_status_word_that_four_bytes_do_not_fit_is_refused():
    c = ref.Case([300, 30], **GQA, seed=5)
    d, dec = device(c), decoder(c)
    new = torch.ones((2, 4, 128), dtype=torch.bfloat16, device=DEV)
    positions = torch.tensor([300, 30], dtype=torch.int32, device=DEV)
    for bad in (torch.zeros(3, dtype=torch.uint8, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV),
                torch.zeros(1, dtype=torch.int32), torch.zeros((4, 4), dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(ValueError):
            dec.append(new, new, positions, d[5], *d[1:5], device_status=bad)
    with pytest.raises(mfa.MfaError):
        dec.append(new, new, positions, d[5], *d[1:5], device_status=torch.zeros(9, dtype=torch.uint8, device=DEV)[1:])
    good = torch.zeros(4, dtype=torch.uint8, device=DEV)
    for word in (good, good.data_ptr()):
        dec.append(new, new, positions + 10 ** 6, d[5], *d[1:5], device_status=word)
    assert int(good.view(torch.int32)) == mfa.MFA_DEV_BAD_LENGTH
