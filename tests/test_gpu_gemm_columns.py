"""The 4-bit GEMM's output columns end at N: whatever N is, the columns of a
wider y and the rows behind its last one stay as they were."""
import pytest
import torch

import nvfp4_w4a4_quantized_09_b200 as nv
from nvfp4_w4a4_quantized_09_b200 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
K = 256


def run(M, N, acts=None):
    """y of `N` of the weight's rows, inside a buffer of sevens."""
    n8 = (N + 7) // 8 * 8
    a = nv.quantize_tensor(synth.student_t_activations(M, K, seed=M, device=DEV))
    w = synth.gaussian_weights(n8, K, 0.05, seed=n8, device=DEV)
    g, _ = nv.global_scale(w)

    def product(n, y):
        codes, sf = nv.quantize(w[:n], g)
        if acts is None:
            nv.gemm(a, nv.QuantizedTensor(codes, sf, g, n, K), y)
        else:
            segments = [(0, n, g)] if n <= 20 else [(0, n - 20, g), (n - 20, 20, g)]
            nv.fused_gemm(a, codes, sf, segments, y, acts=[(acts, None, None)] * len(segments))
    buf = torch.full((M + 1, n8 + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    want = torch.empty(M, n8, dtype=torch.bfloat16, device=DEV)
    product(N, buf[:M, :N])
    product(n8, want)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    return buf, want


@pytest.mark.parametrize("N", [1, 7, 8, 9, 31, 33, 127, 203, 257, 301, 516, 771])
@pytest.mark.parametrize("M", [1, 40, 128, 130, 256, 257, 300, 700])
def test_columns_beyond_n_stay_as_they_were(M, N):
    buf, want = run(M, N)
    assert torch.equal(buf[:M, :N], want[:, :N])
    assert bool((buf[:M, N:] == 7).all()) and bool((buf[M] == 7).all())


@pytest.mark.parametrize("N", [9, 203, 516])
@pytest.mark.parametrize("M", [40, 130, 300])
def test_columns_beyond_n_with_a_gate(M, N):
    buf, want = run(M, N, nv.ACT_SIGMOID)
    assert torch.equal(buf[:M, :N], want[:, :N])
    assert bool((buf[:M, N:] == 7).all()) and bool((buf[M] == 7).all())
