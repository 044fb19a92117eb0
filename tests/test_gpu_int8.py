"""GPU tests of the 8-bit-integer (W8A8) operators: int8_quantize,
add_rms_norm_int8 and int8_gemm against plain references.

Codes, quantizer scales and GEMM outputs are compared bit for bit (their
definitions leave one right value: binary32 steps and exact integer sums); the
norm's scale within the bound that int8_reference.scale_tolerance derives."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int8_reference as ref
import nvfp4_w4a4_quantized_09_b200 as nv
from nvfp4_w4a4_quantized_09_b200 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def f32(t):
    return t.detach().float().cpu().numpy()


def activations(rows, cols, seed):
    return synth.student_t_activations(rows, cols, seed=seed, device=DEV)


def same(got, want):
    """Bit for bit, NaN equal to NaN."""
    return np.array_equal(np.asarray(got), np.asarray(want), equal_nan=True)


# ---------------------------------------------------------------------------
# int8_quantize
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols,pad", [
    (1, 16, 0), (1, 5120, 0), (3, 48, 8), (129, 256, 0), (7, 272, 24), (1001, 512, 0), (5, 4112, 48),
    (2, 8208, 0), (300, 5120, 1000), (8, 17408, 0), (3, 16400, 0), (2, 32768, 0), (2, 32784, 16),
    (2, 70000, 0), (1, 131072, 0)])
def test_quantize_shapes(rows, cols, pad):
    buf = activations(rows, cols + pad, seed=rows + cols)
    x = buf[:, :cols]
    codes, scale = nv.int8_quantize(x)
    torch.cuda.synchronize()
    want_c, want_s = ref.quantize(f32(x))
    assert same(codes.cpu(), want_c) and same(f32(scale), want_s)


def test_quantize_every_finite_bf16_value():
    bits = np.arange(1 << 16, dtype=np.uint32)
    vals = (bits << 16).astype(np.uint32).view(np.float32)
    vals = np.sort(vals[np.isfinite(vals)])
    vals = np.concatenate([vals, np.zeros((-len(vals)) % 64, np.float32)])
    for order in (np.argsort(np.abs(vals), kind="stable"),           # rows of like magnitudes
                  np.random.default_rng(1).permutation(len(vals))):
        x = torch.from_numpy(vals[order].reshape(-1, 64)).to(DEV, BF)
        codes, scale = nv.int8_quantize(x)
        torch.cuda.synchronize()
        want_c, want_s = ref.quantize(f32(x))
        assert same(codes.cpu(), want_c) and same(f32(scale), want_s)


def test_quantize_ties_go_to_the_even_code():
    # max 127 makes the multiplier 1: halves are exact ties
    row = [127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 62.5, 63.5, -62.5, -63.5, 0.0, -0.0, 1.0, 126.5, -126.5]
    codes, scale = nv.int8_quantize(torch.tensor([row], device=DEV, dtype=BF))
    torch.cuda.synchronize()
    assert codes[0].tolist() == [127, 0, 2, 2, 0, -2, -2, 62, 64, -62, -64, 0, 0, 1, 126, -126]
    assert float(scale) == 1.0


def test_quantize_rows_with_nothing_tiny_rows_and_non_finite_rows():
    x = activations(8, 5120, seed=3)
    x[0] = 0
    x[1] = 2.0 ** -110
    x[1, 7] = -2.0 ** -101
    x[2, 5119] = float("nan")
    x[3, 0] = float("inf")
    x[4, 100] = float("-inf")
    x[5] = -0.0
    x[6] = 0
    x[6, 33] = 3.3895313892515355e38
    codes, scale = nv.int8_quantize(x)
    torch.cuda.synchronize()
    want_c, want_s = ref.quantize(f32(x))
    assert same(codes.cpu(), want_c) and same(f32(scale), want_s)
    assert f32(scale)[0] == 1.0 and np.isnan(f32(scale)[2:5]).all() and np.isfinite(f32(scale)[6:]).all()
    assert not codes[2:5].any()


def test_quantize_writes_its_rows_alone():
    x = activations(33, 4112, seed=9)
    codes = torch.full((34, 4112), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((34,), 5.0, device=DEV)
    nv.int8_quantize(x, codes[:33], scale[:33])
    torch.cuda.synchronize()
    want_c, want_s = ref.quantize(f32(x))
    assert same(codes[:33].cpu(), want_c) and same(f32(scale[:33]), want_s)
    assert bool((codes[33] == 77).all()) and float(scale[33]) == 5.0


def test_quantize_empty():
    codes, scale = nv.int8_quantize(torch.empty(0, 64, dtype=BF, device=DEV))
    assert codes.shape == (0, 64) and scale.shape == (0,)


def test_quantize_offsets_beyond_32_bits():
    # rows * stride passes 2^31 elements; codes pass 2^31 bytes in the second
    buf = torch.zeros(33, 1 << 26, dtype=BF, device=DEV)
    x = buf[:, :64]
    x.copy_(activations(33, 64, seed=1))
    codes, scale = nv.int8_quantize(x)
    torch.cuda.synchronize()
    want_c, want_s = ref.quantize(f32(x))
    assert same(codes.cpu(), want_c) and same(f32(scale), want_s)
    del buf, x
    rows = (1 << 31) // 5120 + 3
    x = torch.zeros(rows, 5120, dtype=BF, device=DEV)
    x[-2:] = activations(2, 5120, seed=2)
    codes, scale = nv.int8_quantize(x)
    torch.cuda.synchronize()
    want_c, want_s = ref.quantize(f32(x[-2:]))
    assert same(codes[-2:].cpu(), want_c) and same(f32(scale[-2:]), want_s)
    assert bool((scale[:-2] == 1).all())


# ---------------------------------------------------------------------------
# add_rms_norm_int8
# ---------------------------------------------------------------------------
def norm_inputs(rows, cols, residual, pad, offset, seed):
    x = activations(rows, cols + pad, seed=seed)[:, :cols]
    res = (activations(rows, cols + 2 * pad, seed=seed + 1) * 4)[:, :cols] if residual else None
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (1 - offset + 0.25 * torch.randn(cols, device=DEV, generator=g)).to(BF)
    return x, res, w


def assert_norm(x, res, w, offset, eps, q, res_out):
    codes, scale, v, r = ref.add_rms_norm(f32(x), None if res is None else f32(res), f32(w), offset, eps)
    assert same(q.codes.cpu(), codes)
    s = f32(q.scale).astype(np.float64)
    tol = ref.scale_tolerance(x.shape[1])
    assert np.all(np.abs(s - scale) <= tol * np.abs(scale)), np.max(np.abs(s / scale - 1)) / tol
    if res is None:
        assert res_out is None
    else:
        assert same(f32(res_out), r)
    # each value within half a step of the norm in 64 bits; 127 steps of the
    # scale's own error, and v's roundings (t twice, the multiplier and its
    # product: 4 * 2^-24 of at most 127 steps)
    err = np.abs(codes * s[:, None] - v)
    assert np.all(err <= s[:, None] * (0.5 + 127 * (4 * 2.0 ** -24 + tol)))


@pytest.mark.parametrize("offset", [0.0, 1.0])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1, 16, 0), (2, 48, 8), (1, 5120, 0), (333, 4112, 48),
                                           (65, 512, 0), (700, 5120, 0), (9, 8192, 1000),
                                           (3, 17408, 0), (2, 32784, 0), (2, 66000, 16)])
def test_norm_shapes(rows, cols, pad, residual, offset):
    x, res, w = norm_inputs(rows, cols, residual, pad, offset, seed=rows + cols)
    q, out = nv.add_rms_norm_int8(x, w, residual=res, eps=1e-6, weight_offset=offset)
    torch.cuda.synchronize()
    assert_norm(x, res, w, offset, 1e-6, q, out)


# the last row length of each kernel and the first of the next, several rows a CTA
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(300, 16384, 0), (299, 16400, 8), (330, 17408, 0), (150, 24576, 16),
                                           (151, 24592, 0), (300, 28672, 0), (155, 28688, 0), (149, 32768, 8),
                                           (320, 32784, 0), (149, 51200, 0), (160, 51216, 0)])
def test_norm_long_rows(rows, cols, pad, residual):
    x, res, w = norm_inputs(rows, cols, residual, pad, 1.0, seed=rows + cols)
    q, out = nv.add_rms_norm_int8(x, w, residual=res, weight_offset=1.0)
    torch.cuda.synchronize()
    some = torch.tensor([0, 1, 2, 147, 148, rows - 2, rows - 1], device=DEV)
    assert_norm(x[some], None if res is None else res[some], w, 1.0, 1e-6,
                nv.Int8Tensor(q.codes[some], q.scale[some]), None if res is None else out[some])
    # and every row as if it were alone: the same codes, the same scale
    again, out2 = nv.add_rms_norm_int8(x[3:4], w, residual=None if res is None else res[3:4], weight_offset=1.0)
    assert torch.equal(again.codes[0], q.codes[3]) and torch.equal(again.scale[0], q.scale[3])


@pytest.mark.parametrize("rows,cols", [(160, 40976), (299, 57344), (160, 57360), (149, 102400), (3, 102416)])
def test_quantize_long_rows(rows, cols):
    x = activations(rows, cols, seed=rows)
    codes, scale = nv.int8_quantize(x)
    torch.cuda.synchronize()
    some = torch.tensor([0, 1, rows // 2, rows - 1], device=DEV)
    want_c, want_s = ref.quantize(f32(x[some]))
    assert same(codes[some].cpu(), want_c) and same(f32(scale[some]), want_s)


@pytest.mark.parametrize("cols", [5120, 17408, 33024])
@pytest.mark.parametrize("where", ["residual", "x"])
def test_norm_in_place(where, cols):
    x, res, w = norm_inputs(40, cols, True, 0, 0.0, seed=5)
    x0, res0 = x.clone(), res.clone()
    x, res = x.contiguous(), res.contiguous()
    out = res if where == "residual" else x
    q, got = nv.add_rms_norm_int8(x, w, residual=res, residual_out=out)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    assert_norm(x0, res0, w, 0.0, 1e-6, q, got)


def test_norm_rows_with_nothing_and_non_finite_rows():
    x, res, w = norm_inputs(12, 1024, True, 0, 0.0, seed=8)
    x, res = x.contiguous(), res.contiguous()
    x[0], res[0] = 0, 0
    res[1] = -x[1]                               # cancels to an all-zero row
    x[2, 9] = float("nan")
    res[3, 1023] = float("inf")
    x[4, 3], res[4, 3] = 3e38, 3e38              # the sum is infinite
    x[5] = 3e19                                  # the sum of squares is
    x[6], res[6] = 2.0 ** -100, 0                # far below sqrt(eps)
    x[7], res[7] = 1e-3, 0
    q, out = nv.add_rms_norm_int8(x, w, residual=res)
    torch.cuda.synchronize()
    s = f32(q.scale)
    assert s[0] == 1 and s[1] == 1 and not q.codes[:2].any()
    assert np.isnan(s[2:6]).all() and not q.codes[2:6].any()
    keep = [0, 1, 6, 7, 8, 9, 10, 11]
    assert_norm(x[keep], res[keep], w, 0.0, 1e-6,
                nv.Int8Tensor(q.codes[keep], q.scale[keep]), out[keep])
    _, _, _, r = ref.add_rms_norm(f32(x), f32(res), f32(w), 0.0, 1e-6)
    assert same(f32(out), r)


def test_norm_zero_weight():
    x, res, _ = norm_inputs(3, 256, True, 0, 0.0, seed=8)
    q, _ = nv.add_rms_norm_int8(x, torch.full((256,), -1.0, dtype=BF, device=DEV), residual=res,
                                weight_offset=1.0)
    torch.cuda.synchronize()
    assert not q.codes.any() and bool((q.scale == 1).all())


@pytest.mark.parametrize("eps", [1e-12, 1e-5, 1.0, 1e4])
def test_norm_eps(eps):
    x, res, w = norm_inputs(5, 2048, True, 0, 1.0, seed=2)
    q, out = nv.add_rms_norm_int8(x, w, residual=res, eps=eps, weight_offset=1.0)
    torch.cuda.synchronize()
    assert_norm(x, res, w, 1.0, eps, q, out)


def test_norm_writes_its_rows_alone():
    x, res, w = norm_inputs(21, 5120, True, 8, 0.0, seed=4)
    wide = torch.full((22, 5136), 3.0, dtype=BF, device=DEV)
    codes = torch.full((22, 5120), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((22,), 5.0, device=DEV)
    q, out = nv.add_rms_norm_int8(x, w, residual=res, residual_out=wide[:21, :5120], codes=codes[:21],
                                  scale=scale[:21])
    torch.cuda.synchronize()
    assert_norm(x, res, w, 0.0, 1e-6, q, out)
    assert bool((codes[21] == 77).all()) and float(scale[21]) == 5.0
    assert bool((wide[:, 5120:] == 3).all()) and bool((wide[21] == 3).all())


def test_norm_offsets_beyond_32_bits():
    buf = torch.zeros(33, 1 << 26, dtype=BF, device=DEV)
    out = torch.zeros(33, 1 << 26, dtype=BF, device=DEV)
    x, res, w = norm_inputs(33, 64, True, 0, 0.0, seed=4)
    buf[:, :64] = x
    q, got = nv.add_rms_norm_int8(buf[:, :64], w, residual=res, residual_out=out[:, :64])
    torch.cuda.synchronize()
    assert_norm(x, res, w, 0.0, 1e-6, q, got)
    assert not out[:, 64:72].any()


# ---------------------------------------------------------------------------
# int8_gemm
# ---------------------------------------------------------------------------
def codes(rows, cols, seed, lo=-128, hi=128):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(lo, hi, (rows, cols), device=DEV, generator=g, dtype=torch.int32).to(torch.int8)


def scales(n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.rand(n, device=DEV, generator=g) * 1e-2 + 1e-4


def gemm_inputs(M, N, K, seed=0):
    return (nv.Int8Tensor(codes(M, K, seed + 1), scales(M, seed + 2)),
            nv.Int8Tensor(codes(N, K, seed + 3), scales(N, seed + 4)))


def assert_gemm(a, w, y, rows=slice(None), cols=slice(None)):
    want = ref.gemm(a.codes[rows].cpu().numpy(), f32(a.scale[rows]), w.codes[cols].cpu().numpy(),
                    f32(w.scale[cols]))
    assert same(f32(y[rows][:, cols]), want)


M_SIZES = [1, 2, 3, 8, 9, 15, 16, 17, 31, 32, 33, 48, 64, 65, 100, 128, 129, 200, 255, 256, 257, 300,
           511, 513, 1000]


@pytest.mark.parametrize("N,K", [(5120, 1040), (333, 144), (2051, 16)])
@pytest.mark.parametrize("M", M_SIZES)
def test_gemm_token_counts(M, N, K):
    a, w = gemm_inputs(M, N, K, seed=M)
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    assert_gemm(a, w, y)


@pytest.mark.parametrize("K", [16, 32, 48, 112, 128, 144, 240, 256, 272, 512, 1008, 1024, 1040, 2048,
                               4096, 5120, 17408, 17424])
@pytest.mark.parametrize("M", [1, 37, 130, 260])
def test_gemm_inner_sizes(M, K):
    a, w = gemm_inputs(M, 264, K, seed=K)
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    assert_gemm(a, w, y)


@pytest.mark.parametrize("N", [1, 7, 8, 9, 40, 127, 128, 129, 255, 256, 257, 384, 4096, 18944, 19000])
@pytest.mark.parametrize("M", [1, 20, 140, 290])
def test_gemm_output_widths(M, N):
    a, w = gemm_inputs(M, N, 272, seed=N)
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert y.shape == (M, N) and nv.last_device_status() == 0
    assert_gemm(a, w, y)


@pytest.mark.parametrize("M,N,K", [
    # few tokens: tile widths and stage depths from one step to eight, rounds
    # of tiles, K that ends inside a stage, a step and an instruction
    (128, 24640, 1040), (128, 24640, 1024), (100, 34816, 640), (8, 34816, 1152), (1, 40000, 1280),
    (64, 5120, 1168), (16, 2048, 3200), (33, 151936, 128), (128, 40, 17408),
    # CTA pairs: every tile width, several rounds, bands of M tiles
    (200, 5120, 272), (300, 5120, 272), (200, 24640, 272), (520, 24640, 400), (257, 19000, 144),
    (1000, 5120, 272), (2048, 5120, 144), (260, 151936, 64), (4200, 200, 13008),
    # ... and wide tiles, of both accumulators, N ending in either half
    (1000, 5120, 2608), (200, 24635, 5136), (256, 34816, 4112), (130, 17003, 8192), (700, 4168, 8208),
    (1000, 5120, 17408)])
def test_gemm_configurations(M, N, K):
    a, w = gemm_inputs(M, N, K, seed=M + K)
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    # exact sums in 64 bits, then the three roundings
    acc = a.codes.double() @ w.codes.double().t()
    want = (acc.float() * a.scale[:, None] * w.scale[None, :]).to(BF)
    assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,K", [
    # narrow products of long rows, where the CTAs of a cluster share K: two,
    # four and eight of them, parts of unequal length, N and K that end inside
    # a chunk, a slice, a step and an instruction, M of 1 to 128 MMA rows
    (1, 256, 17408), (3, 169, 27056), (7, 300, 8192), (16, 80, 131056), (20, 6819, 10864), (33, 1024, 28672),
    (34, 1, 10128), (55, 579, 13600), (64, 2051, 8208), (64, 5120, 17408), (65, 80, 22080), (65, 1000, 5136),
    (97, 6738, 19776), (100, 5120, 17408), (104, 4867, 25488), (114, 1111, 2544), (121, 517, 17424),
    (128, 2048, 17408), (128, 8, 131056), (128, 8192, 17408),
    # ... and among CTA pairs, two and four of them, of one M tile and several
    (129, 256, 17408), (160, 2048, 17408), (200, 5120, 17408), (256, 1024, 28672), (256, 2051, 8208),
    (257, 80, 22080), (300, 517, 17424), (384, 5120, 17408), (500, 1000, 5136), (511, 1, 131056),
    (512, 5120, 5120), (700, 300, 27056), (1000, 256, 17408)])
def test_gemm_shares_long_rows_among_ctas(M, N, K):
    a, w = gemm_inputs(M, N, K, seed=M + K)
    y = torch.full((M, (N + 23) // 8 * 8), 7.0, dtype=BF, device=DEV)
    for _ in range(3):
        nv.int8_gemm(a, w, y[:, :N])
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    acc = a.codes.double() @ w.codes.double().t()        # exact
    assert torch.equal(y[:, :N], (acc.float() * a.scale[:, None] * w.scale[None, :]).to(BF))
    assert bool((y[:, N:] == 7).all())


def test_gemm_shared_rows_on_two_streams_and_captured():
    a, w = gemm_inputs(100, 2048, 17408, seed=1)
    b, v = gemm_inputs(40, 300, 28672, seed=2)
    want = nv.int8_gemm(a, w), nv.int8_gemm(b, v)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(nv.int8_gemm(a, w, stream=s), nv.int8_gemm(b, v, stream=s)) for _ in range(10) for s in streams]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(4):
            got.append((nv.int8_gemm(a, w), nv.int8_gemm(b, v)))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    assert all(torch.equal(x, want[0]) and torch.equal(y, want[1]) for x, y in got)


@pytest.mark.parametrize("M,N,K", [(5, 300, 8192), (100, 2048, 17408), (300, 517, 17424)])
def test_gemm_shared_rows_behind_a_long_kernel_and_with_non_finite_scales(M, N, K):
    a, w = gemm_inputs(M, N, K, seed=3)
    want = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    a.scale[M - 1], w.scale[N - 1] = float("nan"), float("inf")
    torch.cuda._sleep(3_000_000_000)                 # about 1.5 s
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    assert bool(y[M - 1].isnan().all()) and not bool(y[:M - 1, N - 1].isfinite().any())
    assert torch.equal(y[:M - 1, :N - 1], want[:M - 1, :N - 1])


@pytest.mark.parametrize("M", [1, 5, 129, 300])
@pytest.mark.parametrize("fill", [(-128, -128), (127, -128), (127, 127)])
def test_gemm_largest_sums(M, fill):
    # |acc| up to 128 * 128 * 131056 = 2^31 - 262144
    K = 131056
    a = nv.Int8Tensor(torch.full((M, K), fill[0], dtype=torch.int8, device=DEV), scales(M, 1))
    w = nv.Int8Tensor(torch.full((300, K), fill[1], dtype=torch.int8, device=DEV), scales(300, 2))
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    want = ref.bf16_round((np.float32(fill[0] * fill[1] * K) * f32(a.scale)[:, None]) * f32(w.scale)[None, :])
    assert same(f32(y), want)


@pytest.mark.parametrize("M", [1, 30, 150, 300])
def test_gemm_one_hot_codes(M):
    # a row with a single one picks one column of the weight: any mistake of
    # layout shows as another integer
    K, N = 400, 260
    a = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    at = (torch.arange(M, device=DEV) * 37 + 11) % K
    a[torch.arange(M, device=DEV), at] = 1
    w = codes(N, K, seed=6)
    one = lambda n: torch.ones(n, device=DEV)  # noqa: E731
    y = nv.int8_gemm(nv.Int8Tensor(a, one(M)), nv.Int8Tensor(w, one(N)))
    torch.cuda.synchronize()
    assert torch.equal(y.float(), w[:, at].t().float())


@pytest.mark.parametrize("M", [1, 17, 200, 300])
def test_gemm_strided_output_and_canary(M):
    N, K = 203, 528
    a, w = gemm_inputs(M, N, K, seed=1)
    buf = torch.full((M + 1, 216), 9.0, dtype=BF, device=DEV)
    nv.int8_gemm(a, w, buf[:M, :N])
    torch.cuda.synchronize()
    assert_gemm(a, w, buf[:M, :N])
    assert bool((buf[:M, N:] == 9).all()) and bool((buf[M] == 9).all())


@pytest.mark.parametrize("M", [1, 17, 200, 300])
def test_gemm_scales_that_are_nan_infinite_zero_or_tiny_stay_in_their_row(M):
    a, w = gemm_inputs(M, 136, 256, seed=3)
    a.scale[M // 2] = float("nan")
    w.scale[5] = float("nan")
    w.scale[6] = float("inf")
    w.scale[7] = 0.0
    w.scale[8] = 1e-38
    w.scale[9] = 1e38
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert_gemm(a, w, y)


@pytest.mark.parametrize("M", [3, 100, 600])
def test_gemm_rows_and_columns_do_not_depend_on_the_rest(M):
    # the same rows alone, and the modules alone, bit for bit
    a, w = gemm_inputs(M, 1500, 2064, seed=7)
    y = nv.int8_gemm(a, w)
    head = nv.int8_gemm(nv.Int8Tensor(a.codes[:2], a.scale[:2]), w)
    parts = [nv.Int8Tensor(w.codes[i:j], w.scale[i:j]) for i, j in ((0, 96), (96, 1000), (1000, 1500))]
    split = torch.cat([nv.int8_gemm(a, p) for p in parts], dim=1)
    fused = nv.int8_gemm(a, nv.Int8Tensor.cat(parts))
    torch.cuda.synchronize()
    assert torch.equal(y[:2], head) and torch.equal(y, split) and torch.equal(y, fused)


def test_gemm_empty():
    a, w = gemm_inputs(4, 8, 32)
    none = nv.Int8Tensor(a.codes[:0], a.scale[:0])
    assert nv.int8_gemm(none, w).shape == (0, 8)
    assert nv.int8_gemm(a, nv.Int8Tensor(w.codes[:0], w.scale[:0])).shape == (4, 0)


@pytest.mark.parametrize("M", [2, 140, 270])
def test_gemm_offsets_beyond_32_bits(M):
    # the weight's codes pass 2^31 bytes
    K = 5120
    N = (1 << 31) // K + 300
    a = nv.Int8Tensor(codes(M, K, 1), scales(M, 2))
    w = nv.Int8Tensor(torch.zeros(N, K, dtype=torch.int8, device=DEV), scales(N, 3))
    w.codes[-290:] = codes(290, K, 4)
    y = nv.int8_gemm(a, w)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    assert_gemm(a, w, y, cols=slice(N - 295, N))
    assert not y[:, :N - 290].any()


@pytest.mark.parametrize("M", [33, 150, 300])
def test_gemm_output_offsets_beyond_32_bits(M):
    a, w = gemm_inputs(M, 40, 64)
    ld = (1 << 31) // (M - 1) // 8 * 8 + 8
    y = torch.zeros(M, ld, dtype=BF, device=DEV)[:, :40]
    nv.int8_gemm(a, w, y)
    torch.cuda.synchronize()
    assert_gemm(a, w, y)


# ---------------------------------------------------------------------------
# together, and how they are called
# ---------------------------------------------------------------------------
def block(x, res, nw, w_qkv, w_gate_up, w_down):
    """One residual block's projections in 8 bits: norm, fused projection; then
    the MLP on the same normed rows and its output back on the stream."""
    q, res = nv.add_rms_norm_int8(x, nw, residual=res, weight_offset=1.0)
    qkv = nv.linear(q, w_qkv)
    out = nv.mlp(q, w_gate_up, w_down)
    return qkv, out, res


@pytest.mark.parametrize("M", [1, 60, 333])
def test_block_runs_together(M):
    H, I = 512, 1152
    x, res, nw = norm_inputs(M, H, True, 0, 1.0, seed=M)
    weights = [synth.gaussian_weights(n, k, 0.02, seed=n, device=DEV) for n, k in ((768, H), (2 * I, H), (H, I))]
    w8 = [nv.int8_quantize_tensor(w) for w in weights]
    qkv, out, r = block(x, res, nw, *w8)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    codes_, scale, v, r_ref = ref.add_rms_norm(f32(x), f32(res), f32(nw), 1.0, 1e-6)
    assert same(f32(r), r_ref)
    # step by step, each operator on the previous one's own output: bit for bit
    q, _ = nv.add_rms_norm_int8(x, nw, residual=res, weight_offset=1.0)
    assert same(q.codes.cpu(), codes_)
    s = f32(q.scale)
    wq = [ref.quantize(f32(w)) for w in weights]
    assert same(f32(qkv), ref.gemm(codes_, s, *wq[0]))
    gu = ref.gemm(codes_, s, *wq[1])
    h = nv.silu_mul(torch.from_numpy(gu).to(DEV, BF))
    hc, hs = ref.quantize(f32(h))
    assert same(f32(out), ref.gemm(hc, hs, *wq[2]))
    # and the projection against the unquantized one in 64 bits: a code is off
    # by half a step (and binary32 roundings far below 2^-13 of one), BF16
    # rounds by 2^-8 relatively
    w64, a64 = f32(weights[0]).astype(np.float64), codes_ * s.astype(np.float64)[:, None]
    y64 = v @ w64.T
    half = 0.5 + 2.0 ** -13
    bound = (half * s[:, None] * np.abs(w64).sum(axis=1)[None, :] +
             half * wq[0][1][None, :] * np.abs(a64).sum(axis=1)[:, None])
    assert np.all(np.abs(f32(qkv) - y64) <= bound + 2.0 ** -8 * (np.abs(y64) + bound))


def test_linear_quantizes_a_bf16_activation():
    x = activations(20, 256, seed=1)
    w = nv.int8_quantize_tensor(synth.gaussian_weights(72, 256, 0.02, seed=2, device=DEV))
    y = nv.linear(x, w)
    torch.cuda.synchronize()
    assert same(f32(y), ref.gemm(*ref.quantize(f32(x)), w.codes.cpu().numpy(), f32(w.scale)))


def test_mlp_mixes_4_and_8_bits():
    x = activations(10, 256, seed=1)
    gate_up = synth.gaussian_weights(512, 256, 0.05, seed=2, device=DEV)
    down = synth.gaussian_weights(256, 256, 0.05, seed=3, device=DEV)
    w4, w8 = nv.quantize_tensor(gate_up), nv.int8_quantize_tensor(down)
    y = nv.mlp(x, w4, w8)
    want = nv.linear(nv.silu_mul(nv.linear(x, w4)), w8)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_mlp_with_an_interleaved_gate_up_takes_an_8_bit_down_projection():
    x = activations(300, 256, seed=1)                # the fused gate_up is for more than 256 tokens
    gate_up = synth.gaussian_weights(512, 256, 0.05, seed=2, device=DEV)
    w4 = nv.quantize_tensor(nv.interleave_gate_up(gate_up))
    w8 = nv.int8_quantize_tensor(synth.gaussian_weights(256, 256, 0.05, seed=3, device=DEV))
    y = nv.mlp(x, w4, w8, interleaved=True)
    h, _, _ = nv.gemm_silu_mul(nv.quantize_tensor(x), w4)
    torch.cuda.synchronize()
    assert same(f32(y), ref.gemm(*ref.quantize(f32(h)), w8.codes.cpu().numpy(), f32(w8.scale)))


@pytest.mark.parametrize("M", [4, 300])
def test_mlp_on_another_stream_keeps_its_intermediates(M):
    # nothing that the call allocated and dropped may be handed out again on
    # the caller's stream while the other one still works on it
    H, I = 256, 512
    x = activations(M, H, seed=1)
    w1 = nv.int8_quantize_tensor(synth.gaussian_weights(2 * I, H, 0.05, seed=2, device=DEV))
    w2 = nv.int8_quantize_tensor(synth.gaussian_weights(H, I, 0.05, seed=3, device=DEV))
    want = nv.mlp(x, w1, w2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)           # some 50 ms
        got = nv.mlp(x, w1, w2, stream=s)
        fill = [torch.full(shape, 0x7F, dtype=torch.int8, device=DEV)
                for shape in ((M, 2 * H), (M, 2 * I), (M, 4 * I), (M, H), (M, I), (4 * M,)) for _ in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del fill


@pytest.mark.parametrize("M", [4, 300])
def test_a_captured_chain_replays_with_new_inputs(M):
    H = 1024
    x, res, nw = norm_inputs(M, H, True, 0, 0.0, seed=1)
    x, res = x.contiguous(), res.contiguous()
    w = nv.int8_quantize_tensor(synth.gaussian_weights(H, H, 0.03, seed=4, device=DEV))

    def chain():
        q, r = nv.add_rms_norm_int8(x, nw, residual=res)
        y = nv.linear(q, w)
        q2, r2 = nv.add_rms_norm_int8(y, nw, residual=r)
        return nv.linear(q2, w), r2

    chain()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for seed in (7, 8, 9):
        x.copy_(activations(M, H, seed=seed))
        torch.cuda.synchronize()
        for _ in range(3):               # both graphs at once
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        want = chain()
        torch.cuda.synchronize()
        for got in outs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert nv.last_device_status() == 0


FIRST_CALL = """
import torch
import nvfp4_w4a4_quantized_09_b200 as nv
for M in (4, 300):
    x = torch.randn(M, 512, device="cuda").bfloat16()
    w = torch.ones(512, device="cuda").bfloat16()
    W = nv.Int8Tensor(torch.randint(-127, 128, (256, 512), device="cuda", dtype=torch.int8),
                      torch.rand(256, device="cuda"))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, r = nv.add_rms_norm_int8(x, w, residual=x)
        y = nv.int8_gemm(q, W)
        c, s = nv.int8_quantize(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, nv.linear(nv.add_rms_norm_int8(x, w, residual=x)[0], W))
    assert torch.equal(c, nv.int8_quantize(x)[0]) and nv.last_device_status() == 0
"""


def test_the_first_call_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]


@pytest.mark.parametrize("M", [2, 140, 270])
def test_calls_on_other_streams(M):
    H = 768
    x, res, nw = norm_inputs(M, H, True, 0, 0.0, seed=1)
    w = nv.int8_quantize_tensor(synth.gaussian_weights(H, H, 0.03, seed=4, device=DEV))
    want = nv.linear(nv.add_rms_norm_int8(x, nw, residual=res)[0], w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(10):
        for s in streams:
            q, _ = nv.add_rms_norm_int8(x, nw, residual=res, stream=s)
            outs.append(nv.linear(q, w, stream=s))
            outs.append(nv.linear(x, w, stream=s)[:0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs if o.shape[0])


@pytest.mark.parametrize("M", [1, 270])
def test_calls_behind_a_long_kernel(M):
    # the kernels are let in early and wait for the previous grid; their bounded
    # waits must not run meanwhile
    H = 512
    x, res, nw = norm_inputs(M, H, True, 0, 0.0, seed=1)
    w = nv.int8_quantize_tensor(synth.gaussian_weights(H, H, 0.03, seed=4, device=DEV))
    want = nv.linear(nv.add_rms_norm_int8(x, nw, residual=res)[0], w)
    torch.cuda.synchronize()
    torch.cuda._sleep(3_000_000_000)                 # about 1.5 s
    got = nv.linear(nv.add_rms_norm_int8(x, nw, residual=res)[0], w)
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0 and torch.equal(got, want)


def test_few_token_and_prefill_products_at_once():
    small, w = gemm_inputs(3, 5120, 2048, seed=1)
    big, _ = gemm_inputs(700, 8, 2048, seed=2)
    want = nv.int8_gemm(small, w), nv.int8_gemm(big, w)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(nv.int8_gemm(small, w, stream=s1), nv.int8_gemm(big, w, stream=s2)) for _ in range(20)]
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in got)


def test_single_rows_of_any_stride_and_refused_strides():
    buf = activations(3, 104, seed=5)
    odd = torch.empty(3 * 100 + 8, dtype=BF, device=DEV)[:300].view(3, 100)
    odd.copy_(buf[:, :100])
    x = odd[:1, :64]                                  # a row stride that is no multiple of 8
    codes_, scale = nv.int8_quantize(x)
    q, r = nv.add_rms_norm_int8(x, torch.ones(64, dtype=BF, device=DEV), residual=x)
    torch.cuda.synchronize()
    want_c, want_s = ref.quantize(f32(x))
    assert same(codes_.cpu(), want_c) and same(f32(scale), want_s)
    assert_norm(x, x, torch.ones(64, dtype=BF), 0.0, 1e-6, q, r)
    for bad in (odd[:2, :64], buf[:1, :64].expand(4, 64), buf[:, 4:68]):
        with pytest.raises(nv.Nvfp4Error):
            nv.int8_quantize(bad)


def test_saved_and_loaded_weight_serves_the_same(tmp_path):
    w = nv.int8_quantize_tensor(synth.gaussian_weights(96, 256, 0.02, seed=2, device=DEV))
    nv.save_quantized(str(tmp_path / "w.pt"), w)
    got = nv.load_quantized(str(tmp_path / "w.pt"))
    x = activations(5, 256, seed=1)
    assert torch.equal(nv.linear(x, got), nv.linear(x, w))
