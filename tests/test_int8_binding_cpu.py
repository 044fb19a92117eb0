"""What the 8-bit calls of the binding do with operands of another kind, without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

import nvfp4_w4a4_quantized_09_b200 as nv


def q8(rows, cols):
    return nv.Int8Tensor(torch.zeros(rows, cols, dtype=torch.int8), torch.ones(rows))


def q4(rows, cols):
    return nv.QuantizedTensor(torch.zeros(rows, cols // 2, dtype=torch.uint8),
                              torch.zeros(nv.sf_bytes(rows, cols), dtype=torch.uint8), torch.ones(1), rows, cols)


@pytest.mark.parametrize("a,w,names", [
    (torch.zeros(4, 64, dtype=torch.int8), q8(8, 64), "Tensor and Int8Tensor"),
    (q8(4, 64), torch.zeros(8, 64, dtype=torch.int8), "Int8Tensor and Tensor"),
    (q8(4, 64), None, "Int8Tensor and NoneType")])
def test_gemm_names_operands_that_are_no_int8_tensors(a, w, names):
    with pytest.raises(TypeError, match=f"two Int8Tensors, not {names}"):
        nv.int8_gemm(a, w)


def test_gemm_refuses_4_bit_operands():
    with pytest.raises(TypeError, match="not QuantizedTensor and Int8Tensor"):
        nv.int8_gemm(q4(4, 64), q8(8, 64))
    with pytest.raises(TypeError, match="not Int8Tensor and QuantizedTensor"):
        nv.int8_gemm(q8(4, 64), q4(8, 64))


WITHOUT_RAW_HANDLES = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import nvfp4_w4a4_quantized_09_b200 as nv


class Stream:
    cuda_stream = 0x50


asked = []
torch.cuda.current_stream = lambda index=None: asked.append(index) or Stream()
assert nv._stream_handle(3, None) == 0x50 and asked == [3]
assert nv._stream_handle(3, Stream()) == 0x50 and asked == [3]
assert nv._current_device is torch.cuda.current_device
"""


def test_streams_are_found_without_torchs_private_handles():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", WITHOUT_RAW_HANDLES], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
