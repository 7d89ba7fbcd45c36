"""The vocabulary loss's bounded waits, without a GPU fault: ufp4_set_quantize_wait_limit(0) makes the first wait for a
stage of every cluster of the products give up at once, with copies in flight into its shared memory.  The kernel
records it, lets the copies land and returns; ufp4_device_error reports it, and the next calls give what they gave
before."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_head_loss_gpu import _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


# single CTAs forward and backward; pairs forward, single CTAs backward; pairs; pairs with several tiles a cluster
@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 1, 8), (16, 5000, 256), (100, 40000, 512), (300, 4000, 512),
                                                 (700, 3000, 1024), (2500, 20000, 128)])
def test_a_wait_that_gives_up_is_reported_and_the_next_call_is_right(tokens, vocab, hidden):
    h, w, t = _inputs(tokens, vocab, hidden, ignored=0.0)
    loss, lse, lse_kept = (torch.empty(tokens, device=DEV) for _ in range(3))
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ws = torch.empty(max(ufp4.ufp4_head_loss_workspace_size(tokens, vocab, hidden),
                         ufp4.ufp4_head_loss_backward_workspace_size(tokens, vocab, hidden)), dtype=torch.uint8, device=DEV)

    def forward(out):
        ufp4.ufp4_head_loss(h, w, t, loss, out, ws)

    def backward():
        ufp4.ufp4_head_loss_backward(h, w, t, lse_kept, dh, dw, ws)
    forward(lse_kept)
    backward()
    torch.cuda.synchronize()
    assert ufp4.ufp4_device_error() == 0
    want = [x.clone() for x in (loss, lse_kept, dh, dw)]
    ufp4.ufp4_set_quantize_wait_limit(0)
    try:
        for call in (lambda: forward(lse), backward):
            call()
            torch.cuda.synchronize()
            assert ufp4.ufp4_device_error_status() == ufp4.UFP4_ERR_TIMEOUT
            assert ufp4.ufp4_device_error() == 0   # the read cleared it
    finally:
        ufp4.ufp4_set_quantize_wait_limit(-1)
    forward(lse)
    backward()
    torch.cuda.synchronize()
    assert ufp4.ufp4_device_error() == 0
    for got, before in zip((loss, lse, dh, dw), want):
        assert torch.equal(got, before)
