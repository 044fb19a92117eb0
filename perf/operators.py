"""Cases for measuring the 8-bit-integer (W8A8) operators.

Three operators, used one after the other in a linear layer that runs in 8-bit
integers beside the 4-bit ones:

* ``add_rms_norm_int8``: residual addition, root-mean-square norm and the
  quantization of the normed row to int8 codes with one FP32 scale per token;
* ``int8_quantize``: int8 codes with one scale per row of a BF16 matrix (an
  activation's token, a weight's output channel);
* ``int8_gemm``: the product of two int8 matrices, accumulated in 32-bit
  integers, scaled per token and per channel and rounded to BF16.

``run`` computes them in elementary torch operations while ``own`` is false and
through the package's entry points while it is true.

The quantizers' result is a pair: int8 codes (the whole numbers they stand for,
in units of the row's scale) and FP32 scales.  Every step that decides a code is
a single binary32 operation, so the codes are one definite set of integers:

    t = fl32(x)                               (int8_quantize)
    r = fl32(x + residual), t = fl32(r * fl32(weight + offset))     (the norm)
    T = max |t| over the row, at least 2^-100
    code = round_half_even(fl32(t * fl32(127 / T)))
    scale = fl32(T / 127)  [times 1 / sqrt(mean(r^2) + eps) for the norm]

(an all-zero row has scale 1).  The norm's factor is common to a row, so it
appears in the scale alone.
"""
import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -100


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step entering a block, hidden size 5120
        {"name": "norm_decode_1x5120", "op": "norm", "rows": 1, "cols": 5120, "residual": True,
         "pad": 0, "offset": 1.0},
        # the first block: no residual yet; a mid-sized ragged batch read out of a wider buffer
        {"name": "norm_first_333x4112_strided", "op": "norm", "rows": 333, "cols": 4112,
         "residual": False, "pad": 48, "offset": 0.0},
        # an 8192-token prefill chunk
        {"name": "norm_prefill_8192x5120", "op": "norm", "rows": 8192, "cols": 5120,
         "residual": True, "pad": 0, "offset": 1.0},
        # a 32K-token prefill
        {"name": "norm_prefill_32768x5120", "op": "norm", "rows": 32768, "cols": 5120,
         "residual": True, "pad": 0, "offset": 0.0},
        # the MLP intermediate of a small decode batch before the down projection
        {"name": "quantize_decode_8x17408", "op": "quantize", "rows": 8, "cols": 17408, "pad": 0},
        # the same of a prefill chunk of odd length
        {"name": "quantize_prefill_8191x17408", "op": "quantize", "rows": 8191, "cols": 17408,
         "pad": 0},
        # a square projection for one token
        {"name": "gemm_decode_1x5120x5120", "op": "gemm", "m": 1, "n": 5120, "k": 5120},
        # gate_up for eight tokens
        {"name": "gemm_decode_8x34816x5120", "op": "gemm", "m": 8, "n": 34816, "k": 5120},
        # the fused input projection for 100 tokens (ragged against every tile)
        {"name": "gemm_decode_100x24640x5120", "op": "gemm", "m": 100, "n": 24640, "k": 5120},
        # the down projection of a short prompt, ragged M
        {"name": "gemm_prompt_1000x5120x17408", "op": "gemm", "m": 1000, "n": 5120, "k": 17408},
        # odd sizes throughout: N not a multiple of 8, K not a multiple of a tile
        {"name": "gemm_ragged_517x2051x1040", "op": "gemm", "m": 517, "n": 2051, "k": 1040},
        # gate_up of an 8192-token prefill chunk
        {"name": "gemm_prefill_8192x34816x5120", "op": "gemm", "m": 8192, "n": 34816, "k": 5120},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "gemm", "gemm"])
    if op == "gemm":
        while True:
            m = _log_int(rng, 1, 16384)
            n = _log_int(rng, 64, 34816)
            k = 16 * _log_int(rng, 8, 1088)
            if m * n * k <= 8192 * 34816 * 5120:
                return {"op": op, "m": m, "n": n, "k": k}
    while True:
        rows = _log_int(rng, 1, 65536)
        cols = 16 * _log_int(rng, 16, 2048)
        if rows * cols <= 8191 * 17408:
            break
    case = {"op": op, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 8, 64, 1000])}
    if op == "norm":
        case["residual"] = rng.random() < 0.75
        case["offset"] = rng.choice([0.0, 1.0])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _student_t(rows, cols, gen, outliers):
    """BF16 heavy-tailed activations (Student-t, 3 degrees of freedom), with a
    few channels far above the others where `outliers`."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    chi = torch.randn(rows, cols, device="cuda", generator=gen).square_()
    for _ in range(2):
        chi += torch.randn(rows, cols, device="cuda", generator=gen).square_()
    x /= chi.div_(3.0).sqrt_()
    if outliers:
        x[:, torch.randperm(cols, device="cuda", generator=gen)[:8]] *= 50.0
    return x.to(torch.bfloat16)


def _strided(x, pad):
    """The same matrix inside a buffer whose rows are `pad` elements longer."""
    if not pad:
        return x
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        a_codes, a_scale = _plain_quantize(_student_t(m, k, gen, outliers=False))
        w = (torch.randn(n, k, device="cuda", generator=gen) * 0.02).to(torch.bfloat16)
        w_codes, w_scale = _plain_quantize(w)
        return {"op": "gemm", "a": (a_codes, a_scale), "w": (w_codes, w_scale)}
    x = _strided(_student_t(case["rows"], case["cols"], gen, outliers=True), case["pad"])
    if case["op"] == "quantize":
        return {"op": "quantize", "x": x}
    # a residual stream some times larger than what a block adds to it, and
    # norm weights around one (kept as they are, or as their offset from one)
    res = None
    if case["residual"]:
        res = torch.randn(case["rows"], case["cols"], device="cuda", generator=gen) * 4.0
        res = _strided(res.to(torch.bfloat16), case["pad"])
    weight = 1.0 + 0.25 * torch.randn(case["cols"], device="cuda", generator=gen)
    return {"op": "norm", "x": x, "residual": res, "offset": case["offset"],
            "weight": (weight - case["offset"]).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def _row_codes(t):
    """(codes, T) of an FP32 matrix: see the module's docstring."""
    amax = t.abs().amax(dim=1, keepdim=True)
    top = amax.clamp_min(TINY)
    codes = torch.round(t * (torch.full_like(top, 127.0) / top)).to(torch.int8)
    return codes, top, amax == 0


def _plain_quantize(x):
    codes, top, zero = _row_codes(x.float())
    scale = torch.where(zero, 1.0, top / torch.full_like(top, 127.0))
    return codes, scale.squeeze(1)


def _plain_norm(x, residual, weight, offset):
    r = x.float() if residual is None else x.float() + residual.float()
    rstd = torch.rsqrt(r.square().mean(dim=1, keepdim=True) + EPS)
    codes, top, zero = _row_codes(r * (weight.float() + offset))
    scale = torch.where(zero, 1.0, top / torch.full_like(top, 127.0) * rstd).squeeze(1)
    return codes, scale, None if residual is None else r.to(torch.bfloat16)


def _plain_gemm(a, w):
    acc = a[0].float() @ w[0].float().t()
    return (acc * a[1][:, None] * w[1][None, :]).to(torch.bfloat16)


def run(state):
    op = state["op"]
    if own:
        import nvfp4_w4a4_quantized_09_b200 as nv
        if op == "gemm":
            (ac, asc), (wc, wsc) = state["a"], state["w"]
            return nv.int8_gemm(nv.Int8Tensor(ac, asc), nv.Int8Tensor(wc, wsc))
        if op == "quantize":
            codes, scale = nv.int8_quantize(state["x"])
            return {"codes": codes, "scale": scale}
        q, res = nv.add_rms_norm_int8(state["x"], state["weight"], residual=state["residual"],
                                      eps=EPS, weight_offset=state["offset"])
        return {"codes": q.codes, "scale": q.scale, "residual": res}
    if op == "gemm":
        return _plain_gemm(state["a"], state["w"])
    if op == "quantize":
        codes, scale = _plain_quantize(state["x"])
        return {"codes": codes, "scale": scale}
    codes, scale, res = _plain_norm(state["x"], state["residual"], state["weight"], state["offset"])
    return {"codes": codes, "scale": scale, "residual": res}


def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 2 * m * n + 4 * (m + n), "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "quantize":
        return {"bytes": rows * cols * 3 + rows * 4, "flops": 4 * rows * cols}
    per = 7 if case["residual"] else 3
    return {"bytes": rows * cols * per + cols * 2 + rows * 4,
            "flops": (8 if case["residual"] else 7) * rows * cols}


def exact(case, seed):
    """The outputs in 64 bits.  The codes are whole numbers that binary32 steps
    decide: they have no other value in 64 bits."""
    state = prepare(case, seed)
    if case["op"] == "gemm":
        (ac, asc), (wc, wsc) = state["a"], state["w"]
        y = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        wide = wc.to(torch.float64)
        for lo in range(0, case["m"], 4096):
            part = torch.mm(ac[lo:lo + 4096].to(torch.float64), wide.t())
            y[lo:lo + 4096] = part * torch.outer(asc[lo:lo + 4096].double(), wsc.double())
        return y
    x = state["x"].double()
    if case["op"] == "quantize":
        return {"codes": None, "scale": x.abs().max(dim=1).values / 127.0}
    if case["residual"]:
        x = x + state["residual"].double()
    biggest = (x * (state["weight"].double() + case["offset"])).abs().max(dim=1).values
    norm = torch.sqrt((x * x).sum(dim=1) / case["cols"] + EPS)
    return {"codes": None, "scale": biggest / 127.0 / norm,
            "residual": x if case["residual"] else None}
