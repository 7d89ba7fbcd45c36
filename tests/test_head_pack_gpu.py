"""The packing of the tokens that have a target, in front of the vocabulary loss's products, on many tokens."""
import pytest
import torch

from rht_bit_block_gb300 import ufp4

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(tokens, seed=1, vocab=8, hidden=8):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.randn((tokens, hidden), generator=g, device=DEV).bfloat16()
    w = torch.randn((vocab, hidden), generator=g, device=DEV).bfloat16()
    t = torch.randint(-1, vocab, (tokens,), generator=g, device=DEV)
    ws = torch.empty(ufp4.ufp4_head_loss_workspace_size(tokens, vocab, hidden), dtype=torch.uint8, device=DEV)
    return h, w, t, torch.empty(tokens, device=DEV), torch.empty(tokens, device=DEV), ws


def _milliseconds(args, repeats=5):
    best = float("inf")
    for _ in range(repeats):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        ufp4.ufp4_head_loss(*args)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_time_goes_with_the_number_of_tokens():
    """Every step of the call is linear in the tokens: four times as many take about four times as long (a count of all
    tokens for each 64 of them would take sixteen times)."""
    few, many = _case(1 << 18), _case(1 << 20)
    times = [_milliseconds(a) for a in (few, many)]
    assert times[1] <= 8 * times[0], times


@pytest.mark.parametrize("tokens", [19455, 19457, 77825, 100003, 200001])
def test_many_tokens(tokens):
    """More tokens than a chunk of rows for each CTA: loss of every token in 64 bits beside it; the gradients are those
    of the tokens with a target alone, and, of h, those of a call on a stretch of the tokens, bit for bit."""
    h, w, t, loss, lse, ws = _case(tokens, seed=tokens)
    ufp4.ufp4_head_loss(h, w, t, loss, lse, ws)
    keep = t >= 0
    logits = h.double() @ w.double().T
    want = torch.logsumexp(logits, 1)
    near = 2.0 ** -19 * (h.double().abs() @ w.double().abs().T).amax(1) + 2.0 ** -20 * (1 + want.abs())
    assert ((lse.double() - want).abs() <= near)[keep].all() and (lse[~keep] == 0).all()
    hit = want - logits.gather(1, t.clamp_min(0)[:, None])[:, 0]
    assert ((loss.double() - hit).abs() <= 2 * near)[keep].all() and (loss[~keep] == 0).all()

    def gradients(rows):
        dh, dw = torch.full_like(h[rows], 7.0), torch.full(tuple(w.shape), 7.0, device=DEV)
        ws = torch.empty(ufp4.ufp4_head_loss_backward_workspace_size(len(dh), 8, 8), dtype=torch.uint8, device=DEV)
        ufp4.ufp4_head_loss_backward(h[rows].contiguous(), w, t[rows].contiguous(), lse[rows].contiguous(), dh, dw, ws)
        return dh, dw
    dh, dw = gradients(slice(None))
    assert (dh[~keep] == 0).all()
    alone = gradients(keep)
    assert torch.equal(dh[keep], alone[0]) and torch.equal(dw, alone[1])
    for stretch in (slice(0, 1000), slice(tokens // 2 - 500, tokens // 2 + 500), slice(tokens - 1000, tokens)):
        assert torch.equal(dh[stretch], gradients(stretch)[0])
    assert ufp4.ufp4_device_error() == 0
