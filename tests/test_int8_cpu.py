"""The 8-bit-integer operators without a GPU: argument checks of the C entry
points and of the binding (all made before anything is enqueued), the
references the GPU tests compare with, and the weight file."""
import ctypes

import numpy as np
import pytest
import torch

import int8_reference as ref
import nvfp4_w4a4_quantized_09_b200 as nv
from nvfp4_w4a4_quantized_09_b200 import _lib, build as _build

OK, ARG, ALIGN, SHAPE = (_lib.NVFP4_OK, _lib.NVFP4_ERR_INVALID_ARG, _lib.NVFP4_ERR_ALIGNMENT,
                         _lib.NVFP4_ERR_UNSUPPORTED_SHAPE)
NUL = 0
A, B, C, D, E = (0x1000000 * i for i in range(1, 6))     # far apart, never dereferenced


@pytest.fixture(scope="module")
def L():
    _build.build()
    return _lib.lib()


def quantize_args(**kw):
    d = dict(x=A, rows=4, cols=64, ld=64, codes=B, scale=C, stream=NUL)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("bad,want", [
    (dict(rows=-1), ARG), (dict(cols=-16), ARG), (dict(cols=24), ALIGN), (dict(ld=68), ALIGN),
    (dict(cols=0, ld=0), SHAPE), (dict(cols=1 << 31, ld=1 << 31), SHAPE), (dict(ld=56), ARG),
    (dict(x=NUL), ARG), (dict(codes=NUL), ARG), (dict(scale=NUL), ARG),
    (dict(x=A + 8), ALIGN), (dict(codes=B + 8), ALIGN), (dict(scale=C + 2), ALIGN),
    (dict(rows=1 << 40, ld=1 << 20), SHAPE), (dict(codes=A + 64), ARG), (dict(scale=A + 16), ARG),
    (dict(scale=B + 252), ARG), (dict(rows=0, x=NUL), OK)])
def test_quantize_refuses(L, bad, want):
    assert L.nvfp4_int8_quantize(*quantize_args(**bad)) == want


def norm_args(**kw):
    d = dict(x=A, ldx=64, residual=B, ldr=64, weight=C, offset=0.0, eps=1e-6, rows=4, cols=64,
             residual_out=D, ldo=64, codes=E, scale=E + 0x100000, stream=NUL)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("bad,want", [
    (dict(rows=-1), ARG), (dict(cols=-16), ARG), (dict(cols=40), ALIGN), (dict(ldx=68), ALIGN),
    (dict(ldr=68), ALIGN), (dict(ldo=68), ALIGN), (dict(ldx=56), ARG), (dict(ldr=56), ARG),
    (dict(ldo=56), ARG), (dict(cols=0), SHAPE), (dict(cols=1 << 31), SHAPE),
    (dict(x=NUL), ARG), (dict(weight=NUL), ARG), (dict(codes=NUL), ARG), (dict(scale=NUL), ARG),
    (dict(residual=NUL), ARG), (dict(x=A + 8), ALIGN), (dict(residual=B + 8), ALIGN),
    (dict(weight=C + 8), ALIGN), (dict(residual_out=D + 8), ALIGN), (dict(codes=E + 8), ALIGN),
    (dict(scale=E + 0x100002), ALIGN), (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(eps=1e-39), ARG),
    (dict(offset=float("nan")), ARG), (dict(offset=float("inf")), ARG), (dict(offset=2.0 ** 100), ARG),
    (dict(offset=-2.0 ** 100), ARG),
    (dict(rows=1 << 40, ldx=1 << 20), SHAPE), (dict(rows=1 << 40, ldr=1 << 20), SHAPE),
    (dict(residual_out=A + 16), ARG), (dict(residual_out=B, ldo=72), ARG), (dict(residual_out=C), ARG),
    (dict(codes=A), ARG), (dict(codes=B), ARG), (dict(codes=C), ARG), (dict(codes=D), ARG),
    (dict(scale=A), ARG), (dict(scale=B), ARG), (dict(scale=C + 64), ARG), (dict(scale=D), ARG),
    (dict(scale=E), ARG), (dict(rows=0, x=NUL), OK)])
def test_norm_refuses(L, bad, want):
    assert L.nvfp4_add_rms_norm_int8(*norm_args(**bad)) == want


def gemm_args(**kw):
    d = dict(a=A, sa=B, w=C, sw=D, y=E, ldy=64, M=4, N=64, K=64, stream=NUL)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("bad,want", [
    (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=-16), ARG), (dict(K=0), SHAPE), (dict(K=24), SHAPE),
    (dict(K=131072), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=1 << 31, ldy=1 << 31), SHAPE),
    (dict(ldy=56), ALIGN), (dict(ldy=68), ALIGN), (dict(M=1 << 30, N=1 << 30, ldy=1 << 30), SHAPE),
    (dict(a=NUL), ARG), (dict(sa=NUL), ARG), (dict(w=NUL), ARG), (dict(sw=NUL), ARG), (dict(y=NUL), ARG),
    (dict(a=A + 8), ALIGN), (dict(w=C + 8), ALIGN), (dict(y=E + 8), ALIGN), (dict(sa=B + 2), ALIGN),
    (dict(sw=D + 2), ALIGN), (dict(y=A + 16), ARG), (dict(y=B), ARG), (dict(y=C), ARG), (dict(y=D), ARG),
    (dict(M=0, a=NUL), OK), (dict(N=0, w=NUL), OK)])
def test_gemm_refuses(L, bad, want):
    assert L.nvfp4_int8_gemm(*gemm_args(**bad)) == want


# ---------------------------------------------------------------------------
# the binding (tensors on the host: each is refused for the reason matched,
# the device last)
# ---------------------------------------------------------------------------
X = torch.zeros(8, 64, dtype=torch.bfloat16)
W = torch.zeros(64, dtype=torch.bfloat16)


def q(rows, cols):
    return nv.Int8Tensor(torch.zeros(rows, cols, dtype=torch.int8), torch.ones(rows))


@pytest.mark.parametrize("call,message", [
    (lambda: nv.int8_quantize(X.float()), "x must be a 2-D bfloat16"),
    (lambda: nv.int8_quantize(X[0]), "x must be a 2-D bfloat16"),
    (lambda: nv.int8_quantize(X.t()), "unit stride"),
    (lambda: nv.int8_quantize(X, codes=torch.zeros(8, 64, dtype=torch.uint8)), "codes must be"),
    (lambda: nv.int8_quantize(X, codes=torch.zeros(8, 32, dtype=torch.int8)), "codes must have shape"),
    (lambda: nv.int8_quantize(X, codes=torch.zeros(64, 8, dtype=torch.int8).t()), "codes must be"),
    (lambda: nv.int8_quantize(X, scale=torch.zeros(7)), "scale must be"),
    (lambda: nv.int8_quantize(X, scale=torch.zeros(8, dtype=torch.float64)), "scale must be"),
    (lambda: nv.int8_quantize(X), "x must be a CUDA tensor"),
    (lambda: nv.add_rms_norm_int8(X, W[:32]), "weight must be"),
    (lambda: nv.add_rms_norm_int8(X, W.float()), "weight must be"),
    (lambda: nv.add_rms_norm_int8(X, W, residual=X[:4]), "residual must have shape"),
    (lambda: nv.add_rms_norm_int8(X, W, residual=X.float()), "residual must be"),
    (lambda: nv.add_rms_norm_int8(X, W, residual_out=X), "residual_out needs a residual"),
    (lambda: nv.add_rms_norm_int8(X, W, residual=X, residual_out=X[:4]), "residual_out must have shape"),
    (lambda: nv.add_rms_norm_int8(X, W, codes=torch.zeros(8, 32, dtype=torch.int8)), "codes must have"),
    (lambda: nv.add_rms_norm_int8(X, W, scale=torch.zeros(9)), "scale must be"),
    (lambda: nv.add_rms_norm_int8(X, W), "x must be a CUDA tensor"),
    (lambda: nv.int8_gemm(q(4, 64), q(8, 32)), "inner dimensions differ"),
    (lambda: nv.int8_gemm(nv.Int8Tensor(q(4, 64).codes, torch.ones(1)), q(8, 64)), "a.scale must be"),
    (lambda: nv.int8_gemm(q(4, 64), nv.Int8Tensor(q(8, 64).codes, torch.ones(4))), "w.scale must be"),
    (lambda: nv.int8_gemm(nv.Int8Tensor(torch.zeros(4, 64), torch.ones(4)), q(8, 64)), "a.codes must be"),
    (lambda: nv.int8_gemm(q(4, 64), q(8, 64), y=torch.zeros(4, 9, dtype=torch.bfloat16)), "y must have"),
    (lambda: nv.int8_gemm(q(4, 64), q(8, 64), y=torch.zeros(4, 8)), "y must be"),
    (lambda: nv.int8_gemm(q(4, 64), q(8, 64)), "a_codes must be a CUDA tensor")])
def test_binding_refuses(call, message):
    with pytest.raises(ValueError, match=message):
        call()


def test_an_int8_activation_needs_an_int8_weight():
    w = nv.QuantizedTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8),
                           torch.ones(1), 4, 64)
    with pytest.raises(TypeError):
        nv.linear(q(2, 64), w)


def test_cat_concatenates_codes_and_scales():
    a, b = q(3, 16), q(5, 16)
    b.scale.fill_(2.0)
    c = nv.Int8Tensor.cat([a, b])
    assert (c.rows, c.cols) == (8, 16) and c.scale.tolist() == [1.0] * 3 + [2.0] * 5


# ---------------------------------------------------------------------------
# the references
# ---------------------------------------------------------------------------
def test_reference_quantizer_is_within_half_a_step_and_uses_the_whole_range():
    rng = np.random.default_rng(0)
    x = ref.bf16_round((rng.standard_t(3, (64, 256)) * np.exp(rng.uniform(-20, 20, (64, 1)))).astype(np.float32))
    codes, scale = ref.quantize(x)
    assert np.all(np.abs(codes).max(axis=1) == 127) and codes.min() >= -127
    # half a step, and the roundings of the multiplier, its product and the
    # scale: 3 * 2^-24 of at most 127 steps
    assert np.all(np.abs(codes * scale.astype(np.float64)[:, None] - x) <=
                  scale[:, None] * (0.5 + 127 * 3 * 2.0 ** -24))


def test_reference_rounding_to_bf16_matches_torch():
    rng = np.random.default_rng(1)
    v = rng.integers(0, 1 << 32, 200000, dtype=np.uint32).view(np.float32)
    want = torch.from_numpy(v.copy()).to(torch.bfloat16).float().numpy()
    assert np.array_equal(ref.bf16_round(v), want, equal_nan=True)


def test_reference_norm_against_64_bits():
    rng = np.random.default_rng(2)
    x = ref.bf16_round(rng.standard_normal((16, 128)).astype(np.float32))
    w = ref.bf16_round(rng.standard_normal(128).astype(np.float32))
    codes, scale, v, r = ref.add_rms_norm(x, x, w, 1.0, 1e-6)
    x64 = 2 * x.astype(np.float64)
    want = x64 / np.sqrt((x64 ** 2).mean(1, keepdims=True) + 1e-6) * (1 + w.astype(np.float64))
    assert np.allclose(v, want, rtol=1e-6)
    assert np.all(np.abs(codes * scale[:, None] - want) <= scale[:, None] * 0.5001)


# ---------------------------------------------------------------------------
# the weight file
# ---------------------------------------------------------------------------
def test_int8_weight_file_round_trip(tmp_path):
    w = nv.Int8Tensor(torch.randint(-127, 128, (6, 32), dtype=torch.int8), torch.rand(6) + 0.1)
    path = str(tmp_path / "w.pt")
    nv.save_quantized(path, w)
    got = nv.load_quantized(path, device="cpu")
    assert isinstance(got, nv.Int8Tensor)
    assert torch.equal(got.codes, w.codes) and torch.equal(got.scale, w.scale)


@pytest.mark.parametrize("change", [
    dict(scale=torch.ones(5)), dict(scale=torch.full((6,), float("nan"))), dict(scale=torch.zeros(6)),
    dict(codes=torch.zeros(6, 32)), dict(codes=torch.zeros(6, 24, dtype=torch.int8))])
def test_int8_weight_file_is_checked(tmp_path, change):
    path = str(tmp_path / "w.pt")
    nv.save_quantized(path, q(6, 32))
    d = torch.load(path, weights_only=True)
    d.update(change)
    torch.save(d, path)
    with pytest.raises(ValueError):
        nv.load_quantized(path, device="cpu")
