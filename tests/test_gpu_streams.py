"""GPU tests of calls on another stream than the current one: what a call
allocates and drops is not handed out again while the other stream works on it."""
import pytest
import torch

import nvfp4_w4a4_quantized_09_b200 as nv
from nvfp4_w4a4_quantized_09_b200 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, I = 256, 512


def delay(stream, cycles=100_000_000):
    """Some 50 ms of one idle thread on `stream`."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(cycles)


def weights():
    gate_up = synth.gaussian_weights(2 * I, H, 0.05, seed=2, device=DEV)
    down = synth.gaussian_weights(H, I, 0.05, seed=3, device=DEV)
    return {"4": (nv.quantize_tensor(gate_up), nv.quantize_tensor(down)),
            "8": (nv.int8_quantize_tensor(gate_up), nv.int8_quantize_tensor(down)),
            "interleaved": (nv.quantize_tensor(nv.interleave_gate_up(gate_up)), None)}


def refill(M):
    """Blocks of every size that an MLP's intermediates may have left behind,
    written over on the current stream."""
    sizes = [4, 512, M * H // 2, M * I // 2, M * H, M * I, 2 * M * H, 2 * M * I, 4 * M * I, 4 * M,
             nv.sf_bytes(M, H), nv.sf_bytes(M, I)]
    return [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]


@pytest.mark.parametrize("M,first,second", [(4, "4", "8"), (300, "4", "8"), (4, "8", "4"), (300, "8", "4"),
                                            (4, "4", "4"), (300, "4", "4"), (300, "interleaved", "8"),
                                            (300, "interleaved", "4")])
def test_mlp_on_another_stream_keeps_its_intermediates(M, first, second):
    x = synth.student_t_activations(M, H, seed=1, device=DEV)
    w = weights()
    args = (x, w[first][0], w[second][1])
    kwargs = {"interleaved": first == "interleaved"}
    s = torch.cuda.Stream()
    nv.mlp(*args, stream=s, **kwargs)
    want = nv.mlp(*args, **kwargs)
    torch.cuda.synchronize()
    for _ in range(3):
        delay(s)
        got = nv.mlp(*args, stream=s, **kwargs)
        kept = refill(M)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del kept
    assert nv.last_device_status() == 0


def test_weights_quantized_on_another_stream():
    mods = [synth.gaussian_weights(n, H, 0.02, seed=n, device=DEV) for n in (128, 64)]
    want = nv.FusedWeight.from_modules(mods)
    want_h = nv.harmonize(want)
    want_kv = nv.kv_quantize(mods[0], nv.kv_scale(mods[0]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        delay(s)
        got = nv.FusedWeight.from_modules(mods, stream=s)
        got_h = nv.harmonize(got, stream=s)
        got_kv = nv.kv_quantize(mods[0], nv.kv_scale(mods[0], stream=s), stream=s)
        kept = refill(128)
        torch.cuda.synchronize()
        assert torch.equal(got.codes, want.codes) and torch.equal(got.sf, want.sf)
        assert all(torch.equal(a, b) for a, b in zip(got.g_list, want.g_list))
        assert torch.equal(got_h.sf, want_h.sf) and torch.equal(got_h.g, want_h.g)
        assert torch.equal(got_kv, want_kv)
        del kept


def test_a_fresh_streams_workspace_is_zeroed_before_its_first_use():
    # the current stream is busy, and the memory a new workspace may get is dirty
    x = synth.student_t_activations(64, H, seed=1, device=DEV)
    want = nv.quantize_tensor(x)
    for _ in range(3):
        dirty = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in (64, 256, 512) for _ in range(8)]
        torch.cuda.synchronize()
        del dirty
        s = torch.cuda.Stream()
        torch.cuda._sleep(100_000_000)
        got = nv.quantize_tensor(x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got.g, want.g) and torch.equal(got.codes, want.codes)


@pytest.mark.parametrize("first,second", [("4", "8"), ("4", "4"), ("interleaved", "8"), ("interleaved", "4")])
def test_two_captured_mlps_replayed_at_once(first, second):
    M = 300
    w = weights()
    kwargs = {"interleaved": first == "interleaved"}
    xs = [synth.student_t_activations(M, H, seed=i, device=DEV) * (1 + 30 * i) for i in range(2)]
    want = [nv.mlp(x, w[first][0], w[second][1], **kwargs) for x in xs]
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([nv.mlp(x, w[first][0], w[second][1], **kwargs) for _ in range(3)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(50):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert nv.last_device_status() == 0
    for outs, right in zip(got, want):
        assert all(torch.equal(o, right) for o in outs)


@pytest.mark.parametrize("M", [5, 300, 5000])
@pytest.mark.parametrize("overlap", [False, True])
def test_host_call_without_a_scratch(M, overlap):
    x = synth.student_t_activations(M, H, seed=1, device=DEV)
    fw = nv.FusedWeight.from_modules([synth.gaussian_weights(n, H, 0.02, seed=n, device=DEV) for n in (256, 64)])
    want = nv.linear(x, fw).cpu()
    x_host = x.cpu().pin_memory()
    y_hosts = [torch.empty(M, fw.rows, dtype=torch.bfloat16).pin_memory() for _ in range(3)]
    s, c = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for kwargs in ({"stream": s}, {}):
        if overlap:
            kwargs["copy_stream"] = c
        for y_host in y_hosts:
            delay(kwargs.get("stream", torch.cuda.current_stream()))
            delay(c)
            nv.linear_host(x_host, fw, y_host, **kwargs)
            kept = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV)
                    for n in (4, 256, 2 * M * fw.rows, 2 * M * H, M * H // 2, nv.sf_bytes(M, H)) for _ in range(3)]
        torch.cuda.synchronize()
        for y_host in y_hosts:
            assert torch.equal(y_host, want)
            y_host.zero_()
        del kept
    assert nv.last_device_status() == 0


def test_streams_by_their_handle_alone():
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    x = synth.student_t_activations(300, H, seed=1, device=DEV)
    w = weights()
    s = torch.cuda.Stream()
    for first, second in (("4", "8"), ("8", "4")):
        want = nv.mlp(x, w[first][0], w[second][1])
        torch.cuda.synchronize()
        delay(s)
        got = nv.mlp(x, w[first][0], w[second][1], stream=Handle(s))
        kept = refill(300)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del kept
    fw = nv.FusedWeight.from_modules([synth.gaussian_weights(64, H, 0.02, seed=1, device=DEV)])
    want = nv.linear(x, fw).cpu()
    x_host, y_host = x.cpu().pin_memory(), torch.empty(300, 64, dtype=torch.bfloat16).pin_memory()
    c = torch.cuda.Stream()
    torch.cuda.synchronize()
    nv.linear_host(x_host, fw, y_host, stream=Handle(s), copy_stream=Handle(c))
    torch.cuda.synchronize()
    assert torch.equal(y_host, want)
