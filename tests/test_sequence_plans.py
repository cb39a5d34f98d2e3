"""What a saved plan of the sequence operators refuses: gradients of a forward
call that its workspace does not hold."""
import pytest
import torch

import recurrent_state_quant_amd as lq


def test_backward_without_a_forward():
    plan = lq.LeapQuantSequence(10, 2, 1, 1, dtype=torch.float32, device="cpu", save=True)
    x, cu = torch.zeros(10, 1, 128), torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(ValueError, match="no forward call"):
        lq.leapquant_sequence_backward(plan, cu, x, x, x, x, x, x, x, x, x, x)
    with pytest.raises(ValueError):  # a refused forward call leaves nothing
        lq.leapquant_sequence_forward(plan, cu, x, x, x, x[..., 0], x[..., 0], x)
    with pytest.raises(ValueError, match="no forward call"):
        lq.leapquant_sequence_backward(plan, cu, x, x, x, x, x, x, x, x, x, x)


@pytest.mark.gpu
def test_backward_of_another_size():
    from tests.test_gpu_sequence import DEV, GRADS, backward, forward, make, offsets
    cu, x = make([70, 30], 1, 2, seed=500)
    plan = lq.LeapQuantSequence(200, 5, 1, 2, dtype=torch.float32, device=DEV, save=True)
    _, d, _, _ = forward(cu, x, 1, 2, plan=plan)
    do = torch.randn((100, 2, 128), generator=torch.Generator().manual_seed(501)).to(DEV)
    first = backward(plan, cu, d, do)
    for at, rows in (([0, 100], 100), ([0, 70, 99], 99), ([0, 70, 70, 100], 100)):
        with pytest.raises(ValueError, match="100 tokens in 2 sequences"):
            backward(plan, at, {m: y[:rows] for m, y in d.items()}, do[:rows])
    # a forward call that is refused changes nothing; one of another size does
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_sequence_forward(plan, offsets([0, 50]), *[d[m][:50] for m in ("q", "k", "v", "beta", "alpha")],
                                      d["v"][:50])
    again = backward(plan, cu, d, do)
    assert all(torch.equal(first[m], again[m]) for m in GRADS)
    forward([0, 5], {m: y[:5] if m != "S0" else y[:2] for m, y in x.items()}, 1, 2, plan=plan)
    with pytest.raises(ValueError, match="5 tokens in 1 sequences"):
        backward(plan, cu, d, do)
