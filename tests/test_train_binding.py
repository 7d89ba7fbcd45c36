"""The binding's operands have to be where the kernels look for them: tensors and checkpoints on the current CUDA
device, workspaces of as many bytes as they say.  No GPU needed: every call here is refused before the library."""
import pytest
import torch

from rht_bit_block_gb300 import build, ufp4

ROWS, COLS, VOCAB = 4, 64, 128


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ufp4.load()


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _ckpt():
    codes, scales = ufp4.alloc_checkpoint(ROWS, COLS, "cpu")
    return ufp4.qtensor(codes, scales, ROWS, COLS)


def _workspace(n=1 << 20):
    return torch.zeros(n, dtype=torch.uint8)


def _calls(ws):
    """Each operator on valid shapes and types, all of it in host memory."""
    m, v, w = _bf16(ROWS, COLS), torch.zeros(ROWS), _bf16(VOCAB, COLS)
    targets, gamma = torch.zeros(ROWS, dtype=torch.int64), torch.ones(COLS)
    return {
        "ufp4_glu": lambda: ufp4.ufp4_glu(m, m, m.clone(), ckpt_gate=_ckpt(), ckpt_up=_ckpt()),
        "ufp4_glu_backward": lambda: ufp4.ufp4_glu_backward(m, _ckpt(), _ckpt(), m.clone(), m.clone(), y=m.clone()),
        "ufp4_rms_norm": lambda: ufp4.ufp4_rms_norm(m, gamma, m.clone(), v, residual=m, total=m.clone(), ckpt=_ckpt()),
        "ufp4_rms_norm_backward": lambda: ufp4.ufp4_rms_norm_backward(m, _ckpt(), v, gamma, m.clone(), gamma.clone(), ws,
                                                                      dtotal=m, y=m.clone()),
        "ufp4_head_loss": lambda: ufp4.ufp4_head_loss(m, w, targets, v, v.clone(), ws),
        "ufp4_head_loss_backward": lambda: ufp4.ufp4_head_loss_backward(m, w, targets, v, m.clone(), w.clone(), ws,
                                                                        token_weight=v, scale=torch.ones(1)),
    }


@pytest.mark.parametrize("name", list(_calls(None)))
def test_host_tensors_are_refused(name, monkeypatch):
    monkeypatch.setattr(ufp4, "_stream", lambda s: 0)          # a host without a GPU has no current stream
    monkeypatch.setattr(ufp4, "load", lambda: pytest.fail("the library was called"))
    with pytest.raises(ValueError, match="host memory"):
        _calls(_workspace())[name]()


class _Elsewhere(torch.Tensor):
    """A tensor that says it is on a device of its own choice."""
    device_index = 0

    def get_device(self):
        return self.device_index


def test_operands_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(ufp4, "_current_device", lambda: 0)
    monkeypatch.setattr(ufp4, "_stream", lambda s: 0)

    def on(device, t):
        t = t.as_subclass(_Elsewhere)
        t.device_index = device
        return t

    def called():
        raise LookupError
    monkeypatch.setattr(ufp4, "load", called)
    m = _bf16(ROWS, COLS)
    with pytest.raises(LookupError):                            # all here: the call goes through
        ufp4.ufp4_glu(on(0, m), on(0, m), on(0, m))
    for k in range(3):
        with pytest.raises(ValueError, match="cuda:1"):
            ufp4.ufp4_glu(*(on(int(i == k), m) for i in range(3)))
    codes, scales = ufp4.alloc_checkpoint(ROWS, COLS, "cpu")
    q = ufp4.qtensor(on(1, codes), on(1, scales), ROWS, COLS)
    with pytest.raises(ValueError, match="cuda:1"):
        ufp4.ufp4_glu(on(0, m), on(0, m), on(0, m), ckpt_gate=q, ckpt_up=q)
    with pytest.raises(ValueError, match="scales"):
        ufp4.qtensor(on(0, codes), on(1, scales), ROWS, COLS)
    with pytest.raises(ValueError, match="host memory"):
        ufp4.ufp4_glu(on(0, m), m, on(0, m))


@pytest.mark.parametrize("name", ["ufp4_rms_norm_backward", "ufp4_head_loss", "ufp4_head_loss_backward"])
def test_workspaces_have_the_bytes_they_count(name, monkeypatch):
    """numel() of an expanded tensor says nothing about its memory."""
    monkeypatch.setattr(ufp4, "_stream", lambda s: 0)
    monkeypatch.setattr(ufp4, "load", lambda: pytest.fail("the library was called"))
    for ws in (_workspace(1).expand(1 << 20), _workspace()[::2]):
        with pytest.raises(ValueError, match="workspace"):
            _calls(ws)[name]()
