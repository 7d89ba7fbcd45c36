"""What an 8-bit checkpoint keeps, by the format itself (tests/train_ref.py, whose bytes the kernels' equal): of an element
v in a block of scale 2^e, 2^-4 of v from 2^(e-6) on, half of the smallest step, 2^(e-10), below.  No GPU needed."""
import torch

from tests import train_ref as ref


def test_error_of_large_and_small_elements():
    g = torch.Generator().manual_seed(1)
    v = torch.randn((400, 320), generator=g) * torch.pow(2.0, torch.randint(-20, 4, (400, 320), generator=g).float())
    v[::3] *= torch.pow(2.0, torch.randint(-40, 40, (v[::3].shape[0], 1), generator=g).float())
    codes, scales = ref.encode(v)
    unit = torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)
    v = v.double()
    err = (ref.decode(codes, scales) - v).abs()
    large = v.abs() >= unit * 2.0 ** -6
    assert large.any() and (~large).any()
    assert (err <= 2.0 ** -4 * v.abs())[large].all()
    assert (err <= 2.0 ** -10 * unit)[~large].all()
    assert (err > 2.0 ** -4 * v.abs())[~large].any()         # there the relative bound does not hold ...
    gone = (codes == 0) & (v != 0)
    assert gone.any() and (v.abs()[gone] <= unit[gone] * 2.0 ** -10).all()   # ... and small elements become 0
