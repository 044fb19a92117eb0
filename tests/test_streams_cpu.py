"""Which stream a call's memory belongs to, without a GPU.

With an explicit stream, everything a call allocates by itself has to come from
that stream's memory: an intermediate that the call drops on return could
otherwise be handed out again on the caller's stream while kernels on the other
one still read or write it.  The library is replaced by one that computes
nothing; what is checked is each allocation and the stream it names."""
import contextlib

import pytest
import torch

import nvfp4_w4a4_quantized_09_b200 as nv

BF = torch.bfloat16
X = torch.zeros(8, 256, dtype=BF)


class Stream:
    cuda_stream = 0x50


S = Stream()


class NoKernels:
    """The library's entry points, none of which does anything but sf_bytes."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        return getattr(self.real, name) if name == "nvfp4_sf_bytes" else lambda *args: 0


def q4(rows, cols):
    return nv.QuantizedTensor(torch.zeros(rows, cols // 2, dtype=torch.uint8),
                              torch.zeros(nv.sf_bytes(rows, cols), dtype=torch.uint8), torch.ones(1), rows, cols)


def q8(rows, cols):
    return nv.Int8Tensor(torch.zeros(rows, cols, dtype=torch.int8), torch.ones(rows))


def fused(cols=256):
    w = q4(96, cols)
    return nv.FusedWeight(w.codes, w.sf, [torch.ones(1), torch.ones(1)], [64, 32], cols)


CALLS = {
    "global_scale": lambda: nv.global_scale(X, stream=S),
    "quantize": lambda: nv.quantize(X, torch.ones(1), stream=S),
    "quantize_tensor": lambda: nv.quantize_tensor(X, stream=S),
    "gemm": lambda: nv.gemm(q4(8, 256), q4(64, 256), stream=S),
    "fused_gemm": lambda: nv.fused_gemm(q4(8, 256), fused().codes, fused().sf, fused().segments(), stream=S),
    "from_modules": lambda: nv.FusedWeight.from_modules([X, X], stream=S),
    "harmonize": lambda: nv.harmonize(fused(), stream=S),
    "silu_mul": lambda: nv.silu_mul(X, stream=S),
    "gemm_silu_mul": lambda: nv.gemm_silu_mul(q4(300, 256), q4(512, 256), stream=S),
    "kv_scale": lambda: nv.kv_scale(X, stream=S),
    "kv_quantize": lambda: nv.kv_quantize(X, torch.ones(1), stream=S),
    "int8_quantize": lambda: nv.int8_quantize(X, stream=S),
    "add_rms_norm_int8": lambda: nv.add_rms_norm_int8(X, X[0], residual=X, stream=S),
    "int8_gemm": lambda: nv.int8_gemm(q8(8, 256), q8(63, 256), stream=S),
    "linear, 4 bits": lambda: nv.linear(X, q4(64, 256), stream=S),
    "linear, fused": lambda: nv.linear(X, fused(), stream=S),
    "linear, 8 bits": lambda: nv.linear(X, q8(64, 256), stream=S),
    "mlp, 4 bits": lambda: nv.mlp(X, q4(512, 256), q4(256, 256), stream=S),
    "mlp, 4 then 8 bits": lambda: nv.mlp(X, q4(512, 256), q8(256, 256), stream=S),
    "mlp, 8 then 4 bits": lambda: nv.mlp(X, q8(512, 256), q4(256, 256), stream=S),
    "mlp, interleaved": lambda: nv.mlp(X, q4(512, 256), q4(256, 256), stream=S, interleaved=True),
    "mlp, interleaved then 8 bits": lambda: nv.mlp(X, q4(512, 256), q8(256, 256), stream=S, interleaved=True),
}


@pytest.mark.parametrize("call", CALLS)
def test_a_call_allocates_on_its_stream_alone(monkeypatch, call):
    real = {name: getattr(torch, name) for name in ("empty", "empty_strided", "empty_like", "zeros")}
    streams, elsewhere = [], []

    def empty(*shape, dtype, device, stream):
        streams.append(stream)
        return real["empty"](*shape, dtype=dtype)

    def other(name):
        def allocate(*args, **kwargs):
            elsewhere.append((name, args))
            return real[name](*args, **kwargs)
        return allocate

    run = CALLS[call]
    workspace, lib = torch.zeros(4096, dtype=torch.uint8), NoKernels(nv._lib.lib())
    monkeypatch.setattr(nv, "_check_devices", lambda **tensors: torch.device("cpu"))
    monkeypatch.setattr(nv, "_workspace", lambda device, stream=None: workspace)
    monkeypatch.setattr(nv._lib, "lib", lambda: lib)
    monkeypatch.setattr(nv, "_empty", empty)
    monkeypatch.setattr(nv, "_on", lambda stream: contextlib.nullcontext(), raising=False)
    inputs = {"q4": q4, "q8": q8, "fused": fused}
    for name, make in inputs.items():        # made before the allocations are watched
        made = {}

        def once(*args, make=make, made=made):
            if args not in made:
                made[args] = make(*args)
            return made[args]
        monkeypatch.setitem(globals(), name, once)
    run()
    streams.clear()
    for name in real:
        monkeypatch.setattr(torch, name, other(name))
    clone = torch.Tensor.clone
    monkeypatch.setattr(torch.Tensor, "clone", lambda t, **kw: elsewhere.append(("clone", t.shape)) or clone(t, **kw))
    run()
    assert not elsewhere
    assert streams and all(s is S for s in streams)


def test_a_scratch_made_by_the_call_belongs_to_both_streams(monkeypatch):
    # the call drops it while both streams still work on it
    class CopyStream:
        cuda_stream = 0x60

    streams, on, recorded, copy = [], [None], [], CopyStream()

    @contextlib.contextmanager
    def enter(stream):
        on.append(stream)
        yield
        on.pop()

    def empty(*shape, dtype, device, stream):
        streams.append(stream)
        return torch.ones(*shape, dtype=dtype)

    zero = torch.Tensor.zero_
    zeroed = []
    w, lib = fused(), NoKernels(nv._lib.lib())
    monkeypatch.setattr(nv, "_check_devices", lambda **tensors: torch.device("cpu"))
    monkeypatch.setattr(nv._lib, "lib", lambda: lib)
    monkeypatch.setattr(nv, "_empty", empty)
    monkeypatch.setattr(nv, "_on", enter)
    monkeypatch.setattr(nv, "_torch_stream", lambda stream: stream, raising=False)
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: zeroed.append((t.numel(), on[-1])) or zero(t))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((tuple(t.shape), s)))
    y_host = torch.empty(8, 96, dtype=BF)
    nv.linear_host(X, w, y_host, stream=S)
    assert len(streams) == 7 and all(s is S for s in streams) and not recorded
    assert zeroed == [(nv._lib.GLOBAL_SCALE_WORKSPACE_BYTES, S)]
    nv.linear_host(X, w, y_host, stream=S, copy_stream=copy)
    assert recorded == [((8, 96), copy)]


def watch_zeros(monkeypatch, capturing):
    """Every torch.zeros call with the stream it is made on (None: the current)."""
    zeros, on, made = torch.zeros, [None], []

    @contextlib.contextmanager
    def enter(stream):
        on.append(stream if stream is not None else on[-1])
        yield
        on.pop()

    def make(*args, **kwargs):
        made.append(on[-1])
        return zeros(*args, dtype=kwargs["dtype"])

    monkeypatch.setattr(nv, "_on", enter, raising=False)
    monkeypatch.setattr(nv, "_workspaces", {})
    monkeypatch.setattr(torch, "zeros", make)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    return made


def test_a_workspace_is_zeroed_on_its_stream_and_kept(monkeypatch):
    made = watch_zeros(monkeypatch, capturing=False)
    dev = torch.device("cuda", 0)
    ws = nv._workspace(dev, S)
    assert made == [S]                       # ordered before the kernel that reads it
    assert nv._workspace(dev, S) is ws and made == [S]


@pytest.mark.parametrize("stream", [None, S])
def test_captured_calls_share_no_workspace(monkeypatch, stream):
    made = watch_zeros(monkeypatch, capturing=True)
    dev = torch.device("cuda", 0)
    a, b = nv._workspace(dev, stream), nv._workspace(dev, stream)
    assert a.data_ptr() != b.data_ptr() and made == [stream] * 2
    assert not nv._workspaces                # nor does a later call outside the graph use them


def test_any_object_with_a_stream_handle_is_a_stream(monkeypatch):
    # as the launches take it: by its cuda_stream
    entered, made = [], []

    class External(torch.cuda.Stream):
        def __new__(cls, handle):
            made.append(handle)
            return object.__new__(Stream)

    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered.append(s) or contextlib.nullcontext())
    with nv._on(S):
        pass
    assert made == [S.cuda_stream] and len(entered) == 1
    with nv._on(None):
        pass
    assert len(entered) == 1
