"""The stream that the sequence operators' calls run on."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from recurrent_state_quant_amd import sequence
from tests.test_gpu_sequence import BF16, DEV, forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [True, False])
def test_current_stream_with_and_without_the_raw_handle(raw, monkeypatch):
    """A call goes to the current stream, whichever way its handle is found."""
    if not raw:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
        monkeypatch.setattr(sequence, "_raw_stream", None)
    else:
        assert sequence._raw_stream is not None
    cu, x = make([150, 40], 2, 4, BF16, seed=510)
    _, _, o, S = forward(cu, x, 2, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _, _, o2, S2 = forward(cu, x, 2, 4)
        y = [torch.empty_like(o2, dtype=torch.float32) for _ in range(2)]
        lq.leapquant_head_norm(o2, o2, *y)
    # whole once that stream alone is waited for
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(*y)
