"""The norm's scale on rows of any length: its error does not grow with them."""
import pytest
import torch

import nvfp4_w4a4_quantized_09_b200 as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16

# u = 2^-24 a rounding.  A thread adds at most 56 squares in one chain of fused
# multiply-adds (rows held on chip: 28672 columns over 512 threads, 51200 over
# 1024), or batches of 32 in binary64 whose total is rounded once: 57 at the
# most.  Two times five shuffle steps join the threads, the mean's factor
# 1 / cols and the addition of eps round once each: (57 + 10 + 2) u.  The inverse
# square root halves that and rounds once; T / 127 and the product round once
# each.  The hundredth covers the products of these.
TOLERANCE = ((57 + 10 + 2) / 2 + 3) * 2.0 ** -24 * 1.01


def check(x, res, weight):
    q, _ = nv.add_rms_norm_int8(x, weight, residual=res, eps=1e-6)
    torch.cuda.synchronize()
    for row in range(x.shape[0]):
        r = x[row].float() if res is None else x[row].float() + res[row].float()
        top = (r * weight.float()).abs().max().double()
        r = r.double()
        want = top / 127 / torch.sqrt(torch.dot(r, r) / x.shape[1] + float(torch.tensor(1e-6)))
        assert abs(float(q.scale[row] / want) - 1) <= TOLERANCE


COLS = [16, 5120, 16400, 28672, 28688, 51200, 51216, 66000, 131072, (1 << 22) + 16, 1 << 25]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols", COLS)
def test_scale_of_random_rows(cols, residual):
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = torch.randn(2, cols, device=DEV, generator=g).to(BF)
    res = (torch.randn(2, cols, device=DEV, generator=g) * 4).to(BF) if residual else None
    w = (1 + 0.25 * torch.randn(cols, device=DEV, generator=g)).to(BF)
    check(x, res, w)


@pytest.mark.parametrize("value", [1.296875, 0.69921875, 1.09375, 3.09375])
@pytest.mark.parametrize("cols", COLS)
def test_scale_of_constant_rows(cols, value):
    # every rounding of a chain of equal squares falls the same way for long
    # stretches: the errors add up
    x = torch.full((1, cols), value, device=DEV, dtype=BF)
    res = torch.full((1, cols), value * 2.0 ** -9, device=DEV, dtype=BF)
    w = torch.ones(cols, device=DEV, dtype=BF)
    check(x, None, w)
    check(x, res, w)
