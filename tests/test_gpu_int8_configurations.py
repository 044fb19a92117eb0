"""The int8 GEMM in every form that its launcher chooses, bit for bit, and the
row kernels on both sides of each switch between them."""
import numpy as np
import pytest
import torch

import int8_reference as ref
import nvfp4_w4a4_quantized_09_b200 as nv
from nvfp4_w4a4_quantized_09_b200 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def operand(rows, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(-128, 128, (rows, cols), device=DEV, generator=g, dtype=torch.int32).to(torch.int8)
    return nv.Int8Tensor(codes, torch.rand(rows, device=DEV, generator=g) * 1e-2 + 1e-4)


def assert_product(M, N, K):
    """Three products into the first N columns of a wider buffer of sevens."""
    a, w = operand(M, K, seed=M + K), operand(N, K, seed=N)
    buf = torch.full((M + 1, (N + 23) // 8 * 8), 7.0, dtype=BF, device=DEV)
    for _ in range(3):
        nv.int8_gemm(a, w, buf[:M, :N])
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    acc = a.codes.double() @ w.codes.double().t()                # exact
    assert torch.equal(buf[:M, :N], (acc.float() * a.scale[:, None] * w.scale[None, :]).to(BF))
    assert bool((buf[:M, N:] == 7).all()) and bool((buf[M] == 7).all())


# Channels as the MMA's rows: 1 to 32 tokens on 33152 channels and more, in one and
# two chunks of 16 tokens; K of whole steps, ending inside a step, inside an
# instruction and inside the first step; N ending inside a tile.
@pytest.mark.parametrize("K", [16, 128, 400, 1168, 1280, 5120])
@pytest.mark.parametrize("M,N", [(1, 33152), (15, 33157), (16, 33280), (17, 33160), (24, 34816), (31, 33153),
                                 (32, 34816), (32, 40003)])
def test_swapped_products(M, N, K):
    assert_product(M, N, K)


# One shape or more for each of the other few-token forms on 148 SMs: whole tiles and
# K shared by 2, 4 and 8 CTAs, with 1, 2, 4 and 8 k-steps a stage.
@pytest.mark.parametrize("M,N,K", [
    (26, 31022, 128), (125, 20535, 800), (97, 1, 128), (83, 5858, 48), (41, 1, 128), (64, 102, 224), (1, 1, 128),
    (13, 56, 256), (32, 33151, 1040),
    (123, 7175, 3552), (125, 9869, 18064), (98, 1, 2208), (29, 6329, 19584), (74, 1, 2592), (42, 3377, 6368),
    (1, 2668, 3312), (8, 2970, 3728), (1, 2720, 5120), (8, 2720, 5120),
    (124, 3557, 3904), (114, 3727, 18864), (49, 1, 2896), (62, 72, 7936), (1, 1, 2608), (19, 84, 4048),
    (105, 1, 10224), (113, 63, 15792), (1, 1, 8784), (81, 14, 26544)])
def test_few_token_products(M, N, K):
    assert_product(M, N, K)


# The same for CTA pairs: narrow and wide tiles and K shared by two and four
# pairs, of every width.
@pytest.mark.parametrize("M,N,K", [
    (132, 1, 128), (132, 4942, 128), (266, 3891, 128), (135, 9750, 128), (258, 5983, 128), (288, 7355, 128),
    (293, 17264, 128), (522, 3341, 736), (332, 39458, 1248),
    (257, 10833, 400), (793, 4965, 608), (130, 26032, 816), (257, 14917, 1184), (260, 16854, 1776),
    (1683, 3441, 4864),
    (3872, 1, 1504), (263, 1096, 2032), (260, 1546, 2624), (4143, 132, 3360), (260, 2865, 4160), (280, 3270, 5296),
    (4127, 235, 7392), (1274, 871, 6512), (184, 6585, 13008),
    (132, 1, 1296), (1813, 67, 2336), (268, 701, 3920), (1985, 133, 5760), (260, 1154, 7200), (259, 1537, 9616),
    (264, 1636, 13760), (154, 1369, 3872), (138, 2424, 19472)])
def test_pair_products(M, N, K):
    assert_product(M, N, K)


# the last row length of each form of the plain quantizer and the first of the
# next, several rows a CTA
@pytest.mark.parametrize("rows,cols", [(700, 12288), (700, 12304), (401, 20480), (401, 20496), (400, 40960),
                                       (300, 40976), (299, 57344), (150, 57360), (149, 102400), (149, 102416)])
def test_quantizer_switches(rows, cols):
    x = synth.student_t_activations(rows, cols, seed=rows, device=DEV)
    codes, scale = nv.int8_quantize(x)
    torch.cuda.synchronize()
    some = torch.tensor([0, 1, 147, 148, rows // 2, rows - 1], device=DEV)
    want_c, want_s = ref.quantize(x[some].float().cpu().numpy())
    assert np.array_equal(codes[some].cpu().numpy(), want_c)
    assert np.array_equal(scale[some].cpu().numpy(), want_s)
    # every row as if it were alone, in steps that one binary32 rounding decides
    top = x.abs().amax(dim=1).float()
    assert torch.equal(scale, top / torch.full_like(top, 127.0))
    mult = torch.full_like(top, 127.0) / top
    for lo in range(0, rows, 64):
        assert torch.equal(codes[lo:lo + 64], torch.round(x[lo:lo + 64].float() * mult[lo:lo + 64, None]).to(torch.int8))


@pytest.mark.parametrize("offset", [-1.0, 0.3, 2.5, -2.0 ** 20])
@pytest.mark.parametrize("rows,cols,residual", [(3, 512, True), (3, 512, False), (200, 24592, True),
                                                (2, 51216, True)])
def test_norm_weight_offsets(rows, cols, residual, offset):
    # t = fl32(r * fl32(w + offset)), whatever the offset
    x = synth.student_t_activations(rows, cols, seed=1, device=DEV)
    res = synth.student_t_activations(rows, cols, seed=2, device=DEV) if residual else None
    g = torch.Generator(device=DEV).manual_seed(cols)
    w = (0.5 * torch.randn(cols, device=DEV, generator=g)).to(BF)
    q, out = nv.add_rms_norm_int8(x, w, residual=res, weight_offset=offset)
    torch.cuda.synchronize()
    f32 = lambda t: None if t is None else t[:3].float().cpu().numpy()  # noqa: E731
    codes, scale, _, r = ref.add_rms_norm(f32(x), f32(res), w.float().cpu().numpy(), offset, 1e-6)
    assert np.array_equal(q.codes[:3].cpu().numpy(), codes)
    assert np.all(np.abs(q.scale[:3].double().cpu().numpy() / scale - 1) <= ref.scale_tolerance(cols))
    assert out is None if res is None else np.array_equal(f32(out), r)
