"""The vocabulary loss's gradients on both sides of the rule that gives few tokens' dl to single CTAs or to pairs: it
looks at the tokens (tiles of 128) and, for two such tiles, at the vocabulary.  Tolerances: tests/test_head_loss_gpu.py."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4
from tests.test_head_loss_gpu import _backward, _check_backward, _check_forward, _forward, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [128, 129, 256, 257, 384, 385])
@pytest.mark.parametrize("vocab", [100000, 100001, 131072])
def test_either_side_of_the_rule(tokens, vocab):
    h, w, t = _inputs(tokens, vocab, 72, seed=tokens, ignored=0.1)
    loss, lse = _forward(h, w, t)
    _check_forward(h, w, t, loss, lse)
    dh, dw = _backward(h, w, t, lse)
    _check_backward(h, w, t, dh, dw)


def test_the_vocabulary_beside_a_token_changes_only_its_own_columns():
    """Entries of w that no logit comes near (their rows are far below) carry no gradient to the rest: a call whose
    vocabulary crosses the rule's limit by such rows gives the other rows of dw the bits of the smaller call."""
    tokens, vocab, hidden = 200, 100000, 64
    h, w, t = _inputs(tokens, vocab + 1, hidden, seed=3, ignored=0.0)
    t.clamp_max_(vocab - 1)
    h, w = h.contiguous(), w.contiguous()
    h[:, 0] = 4.0
    w[vocab] = 0
    w[vocab, 0] = -256.0                                     # its logits are -1024: exp is 0 beside the others
    lse = _forward(h, w[:vocab], t)[1]
    few, many = _backward(h, w[:vocab], t, lse), _backward(h, w, t, lse)
    assert torch.equal(few[1], many[1][:vocab]) and (many[1][vocab] == 0).all()
    assert ufp4.ufp4_device_error() == 0
