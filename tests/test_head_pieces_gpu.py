"""The vocabulary loss's gradients over several pieces of the vocabulary: dH added up across launches or in shares of
every piece, the two buffers of dl used in turn, dW of pieces that do not begin at the vocabulary's first row.

Tolerances are those of tests/test_head_loss_gpu.py: an entry within 2^-8 (1 + 2^-4) of the sum of magnitudes, the
difference's 2-norm within 2^-8 of the result's."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_head_loss_gpu import _backward, _check_backward, _check_forward, _forward, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _pieces_and_shares(tokens, vocab, hidden):
    """At least how many pieces, and how many fp32 sums of dH, a workspace of the size asked for can stand for: it holds
    dl (bf16) of two pieces, the packed rows of h, the sums, and less than one sum's bytes beside them."""
    ws = ufp4.ufp4_head_loss_backward_workspace_size(tokens, vocab, hidden)
    rows, cols = -(-tokens // 256) * 256, -(-hidden // 8) * 8
    assert ws < 2 * rows * vocab                                  # the whole dl does not fit
    pieces = next(n for n in range(2, 1000) if ws >= 4 * rows * (vocab // n // 256 * 256) + 2 * rows * cols)
    piece = -(-(-(-vocab // pieces)) // 256) * 256
    return pieces, (ws - 4 * rows * piece - 2 * rows * cols) // (4 * rows * cols)


# tokens, vocabulary, hidden; pieces at least; dH in shares of its own
CASES = [(20000, 20001, 72, 3, False), (33000, 10001, 520, 3, False), (12000, 40000, 64, 3, True),
         (2300, 200001, 64, 3, True)]


@pytest.mark.parametrize("tokens,vocab,hidden,pieces,shared", CASES)
def test_gradients_over_several_pieces(tokens, vocab, hidden, pieces, shared):
    found, shares = _pieces_and_shares(tokens, vocab, hidden)
    assert found >= pieces and (shares > found if shared else shares == 1), (found, shares)
    h, w, t = _inputs(tokens, vocab, hidden, seed=vocab, ignored=0.05)
    # targets at both ends of every piece's range, wherever the pieces lie: each multiple of 256 and its neighbours
    edges = torch.cat([torch.arange(0, vocab, 256, device=DEV) + i for i in (-1, 0, 1)])
    edges = torch.cat([edges[(edges >= 0) & (edges < vocab)], torch.tensor([vocab - 1], device=DEV)])
    t[:len(edges)] = edges[:tokens]
    g = torch.Generator(device=DEV).manual_seed(1)
    weight = 0.5 + torch.rand((tokens,), generator=g, device=DEV)
    scale = torch.full((1,), 1.0 / tokens, device=DEV)
    z = 1e-4
    loss, lse = _forward(h, w, t, z)
    _check_forward(h, w, t, loss, lse, z)
    dh, dw = _backward(h, w, t, lse, weight, scale, z, torch.float32, torch.float32)
    _check_backward(h, w, t, dh, dw, weight, scale, z)
    # one gradient at a time, and bf16 outputs: the same sums
    only, _ = _backward(h, w, t, lse, weight, scale, z, torch.bfloat16, None)
    assert torch.equal(only, dh.bfloat16())
    _, only = _backward(h, w, t, lse, weight, scale, z, None, torch.bfloat16)
    assert torch.equal(only, dw.bfloat16())
    # added to what is there, every piece's rows
    start = torch.randn((vocab, hidden), generator=g, device=DEV)
    total = start.clone()
    ws = torch.full((ufp4.ufp4_head_loss_backward_workspace_size(tokens, vocab, hidden),), 255, dtype=torch.uint8, device=DEV)
    ufp4.ufp4_head_loss_backward(h, w, t, lse, None, total, ws, token_weight=weight, scale=scale, z_loss=z, accumulate_dw=True)
    assert torch.equal(total, start + dw)
    assert ufp4.ufp4_device_error() == 0
