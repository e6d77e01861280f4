"""What the Python binding of the paged and rotary calls does besides passing arguments on."""
import pytest
import torch

import decode_attention_11_b200 as tq

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def keep_busy(stream, n=60):
    """Some tens of milliseconds of work on `stream`."""
    with torch.cuda.stream(stream):
        a = torch.ones(8192, 8192, device="cuda", dtype=torch.bfloat16)
        b = torch.empty_like(a)
        for _ in range(n):
            torch.mm(a, a, out=b)


def test_check_sees_calls_on_every_stream():
    pt = tq.PageTable.allocate(2, 4, 8, 16)
    seqs, one, far = ints([0]), ints([1]), ints([7])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        keep_busy(side)
        tq.pages_reserve(pt, far, one, 1, stream=side)  # no such sequence: recorded when the stream gets there
        with pytest.raises(ValueError, match="out of range"):
            pt.check()
        pt.check()
        # what is recorded right after a check that clears is not lost
        keep_busy(torch.cuda.current_stream(), 5)
        tq.pages_reserve(pt, far, one, 1)
        with pytest.raises(ValueError, match="out of range"):
            pt.check()
        tq.pages_free(pt, far, stream=side)
        with pytest.raises(ValueError, match="out of range"):
            pt.check()
    assert tq.pages_reserve(pt, seqs, one, 1).tolist() == [0]
    pt.check()
