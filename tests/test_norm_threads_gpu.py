"""The norm's passes called from several host threads at once, at widths that share a kernel but not its shared
memory: every call is valid, so every call succeeds, with the results of a call made alone."""
import ctypes
import threading

import pytest
import torch

from rht_bit_block_gb300 import ufp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
CALLS = 3000


class Work:
    """Operands of one thread: forward and backward passes of `rows` rows, fp32 inputs."""

    def __init__(self, rows, cols, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.shape = rows, cols
        self.x = torch.randn((rows, cols), generator=g, device=DEV)
        self.dy = torch.randn((rows, cols), generator=g, device=DEV)
        self.gamma = 1 + 0.1 * torch.randn((cols,), generator=g, device=DEV)
        self.codes, self.scales = ufp4.alloc_checkpoint(rows, cols, DEV)
        self.q = ufp4.qtensor(self.codes, self.scales, rows, cols)
        self.y, self.dx = (torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.rstd, self.dgamma = torch.zeros(rows, device=DEV), torch.zeros(cols, device=DEV)
        self.ws = torch.empty(ufp4.ufp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=DEV)

    def results(self):
        return [t.clone() for t in (self.y, self.rstd, self.codes, self.scales, self.dx, self.dgamma)]

    def calls(self, stream):
        """Both passes as argument tuples of the C entries: a loop over them spends its time in the library."""
        rows, cols = self.shape
        q, n = ctypes.byref(self.q), self.ws.numel()
        forward = (self.x.data_ptr(), cols, ufp4.F32, None, 0, self.gamma.data_ptr(), ufp4.F32, rows, cols, 1e-6,
                   self.y.data_ptr(), cols, None, 0, self.rstd.data_ptr(), q, stream)
        backward = (self.dy.data_ptr(), cols, ufp4.F32, q, self.rstd.data_ptr(), self.gamma.data_ptr(), ufp4.F32, None, 0,
                    rows, cols, self.dx.data_ptr(), cols, self.dgamma.data_ptr(), None, 0, self.ws.data_ptr(), n, stream)
        return forward, backward


@pytest.mark.parametrize("widths", [(2048, 5000), (9216, 20480)])
def test_norm_from_several_host_threads(widths):
    lib = ufp4.load()
    work = [Work(3, cols, i) for i, cols in enumerate(widths * 2)]
    alone = []
    for w in work:
        forward, backward = w.calls(torch.cuda.current_stream().cuda_stream)
        assert lib.ufp4_rms_norm(*forward) == 0 and lib.ufp4_rms_norm_backward(*backward) == 0
        torch.cuda.synchronize()
        alone.append(w.results())
        for t in (w.y, w.dx, w.rstd, w.dgamma, w.codes, w.scales):
            t.zero_()
    torch.cuda.synchronize()
    barrier = threading.Barrier(len(work))
    statuses = [None] * len(work)

    def run(i):
        s = torch.cuda.Stream()
        forward, backward = work[i].calls(s.cuda_stream)
        bad = 0
        barrier.wait(timeout=60)
        for _ in range(CALLS):
            bad += lib.ufp4_rms_norm(*forward) != 0
            bad += lib.ufp4_rms_norm_backward(*backward) != 0
        s.synchronize()
        statuses[i] = bad

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert statuses == [0] * len(work), f"calls that failed, of {2 * CALLS} a thread: {statuses}"
    for w, want in zip(work, alone):
        for a, b in zip(w.results(), want):
            assert torch.equal(a, b)
