"""Measured cases of the RMS norm with an 8-bit output and of the int8 operators.

Four operators, each in its plain form (elementary torch operations) and, with
`own` set, as a user calls the library:

  norm      native.rms_norm_quantize  residual addition, RMS norm, the result as E4M3
                                      codes (a scale per 128 columns), as int8 codes (a
                                      scale per token), in bf16 or f32
  quantize  native.int8_quantize      int8 codes and one fp32 scale per row (a token of
                                      activations, an output channel of a weight)
  linear    native.int8_linear        y = x . W^T on such operands
  mlp       native.int8_mlp           gated MLP with int8 weights, x and h quantised per
                                      token
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
INT8_MAX = 127.0
TINY = 2.0 ** -126
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token between two blocks, into FP8 projections (a latency-bound call)
        dict(name="norm T1 5120 fp8", op="norm", T=1, H=5120, x="bf16", res="bf16", w="bf16",
             codes="fp8", y=""),
        # a decode batch in front of an MoE layer: bf16 for the router, int8 for the experts
        dict(name="norm T16 2048 int8 and bf16", op="norm", T=16, H=2048, x="bf16", res="bf16",
             w="bf16", codes="int8", y="bf16"),
        # a ragged batch on an fp32 residual stream, last block of 32 columns
        dict(name="norm T333 1056 fp8, f32 stream", op="norm", T=333, H=1056, x="bf16", res="f32",
             w="f32", codes="fp8", y=""),
        # a prefill chunk in front of int8 projections
        dict(name="norm T2048 5120 int8", op="norm", T=2048, H=5120, x="bf16", res="bf16",
             w="bf16", codes="int8", y=""),
        # a decode batch's activations in front of a down projection (long rows)
        dict(name="quantize act 16x17408", op="quantize", rows=16, cols=17408, dtype="bf16"),
        # a checkpoint's fp32 MLP matrix turned into int8 weights
        dict(name="quantize weight 17408x5120", op="quantize", rows=17408, cols=5120, dtype="f32"),
        # one token through the widest projection of a dense block
        dict(name="linear M1 17408x5120", op="linear", M=1, N=17408, K=5120, pre=False, out="bf16"),
        # a decode batch through a short projection with a long K, codes already made
        dict(name="linear M24 5120x17408", op="linear", M=24, N=5120, K=17408, pre=True,
             out="bf16"),
        # a ragged batch: N no multiple of a tile, K no multiple of 128, fp32 out
        dict(name="linear M77 5000x2080", op="linear", M=77, N=5000, K=2080, pre=False, out="f32"),
        # a prefill chunk on operands quantised once for several projections
        dict(name="linear M2048 17408x5120", op="linear", M=2048, N=17408, K=5120, pre=True,
             out="bf16"),
        # a few users' tokens through a dense int8 MLP block
        dict(name="mlp T4 5120x17408", op="mlp", T=4, H=5120, I=17408, pre=False),
        # a prefill chunk through it, x from the norm in codes
        dict(name="mlp T512 5120x17408", op="mlp", T=512, H=5120, I=17408, pre=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "linear", "linear", "mlp"])
    if op == "norm":
        codes = rng.choice(["fp8", "int8", "int8", ""])
        return dict(op=op, T=_log_int(rng, 1, 4096), H=_log_int(rng, 32, 8192, 32),
                    x=rng.choice(["bf16", "bf16", "f32"]), res=rng.choice(["", "bf16", "f32"]),
                    w=rng.choice(["bf16", "f32"]), codes=codes,
                    y=rng.choice(["", "bf16", "f32"]) if codes else rng.choice(["bf16", "f32"]))
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, 4096), cols=_log_int(rng, 32, 17408, 32),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        K = _log_int(rng, 32, 17408, 32)
        return dict(op=op, M=min(_log_int(rng, 1, 2048), 2048 * 5120 // K),
                    N=_log_int(rng, 17, 17408) if K <= 5120 else _log_int(rng, 17, 5120), K=K,
                    pre=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    return dict(op=op, T=_log_int(rng, 1, 512), H=_log_int(rng, 256, 5120, 32),
                I=_log_int(rng, 96, 17408, 32), pre=rng.random() < 0.5)


def _blocks(n):
    return -(-n // BLOCK)


def _size(t):
    return {"": 0, "bf16": 2, "f32": 4}[t]


def work(c):
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        per = _size(c["x"]) + 2 * _size(c["res"]) + _size(c["y"]) + (1 if c["codes"] else 0)
        scales = {"": 0, "int8": 1, "fp8": _blocks(c["H"])}[c["codes"]] * c["T"]
        return {"bytes": n * per + c["H"] * _size(c["w"]) + 4 * scales, "flops": 6 * n}
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (_size(c["dtype"]) + 1) + 4 * c["rows"], "flops": 3 * n}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        x = M * K + 4 * M if c["pre"] else 2 * M * K
        return {"bytes": x + N * K + 4 * N + M * N * _size(c["out"]), "flops": 2 * M * N * K}
    T, H, I = c["T"], c["H"], c["I"]
    x = T * H + 4 * T if c["pre"] else 2 * T * H
    return {"bytes": 3 * H * I + 4 * (2 * I + H) + x + 2 * T * H, "flops": 6 * T * H * I}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _acts(g, rows, cols):
    """Activations with channels of different strength, as in front of a projection."""
    strength = torch.exp(0.5 * _randn(g, 1, cols))
    return _randn(g, rows, cols) * strength


def _int8_weight(g, n, k):
    """codes int8 [n, k] and scales f32 [n] of N(0, 0.02) weights."""
    return _int8_plain(_randn(g, n, k, std=0.02))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["rows"] = _acts(g, T, H).to(TYPES[case["x"]])
        s["residual"] = _acts(g, T, H).mul_(4.0).to(TYPES[case["res"]]) if case["res"] else None
        s["weight"] = (1.0 + _randn(g, H, std=0.2)).to(TYPES[case["w"]])
    elif case["op"] == "quantize":
        weight = case["dtype"] == "f32"
        x = _randn(g, case["rows"], case["cols"], std=0.02) if weight else \
            _acts(g, case["rows"], case["cols"])
        s["x"] = x.to(TYPES[case["dtype"]])
    else:
        mlp = case["op"] == "mlp"
        rows, cols = (case["T"], case["H"]) if mlp else (case["M"], case["K"])
        s["x"], s["xs"] = _acts(g, rows, cols).to(torch.bfloat16), None
        if case["pre"]:
            s["x"], s["xs"] = _int8_plain(s["x"])
        if mlp:
            for name, n, k in (("gate", case["I"], case["H"]), ("up", case["I"], case["H"]),
                               ("down", case["H"], case["I"])):
                s[name] = _int8_weight(g, n, k)
        else:
            s["w"], s["ws"] = _int8_weight(g, case["N"], case["K"])
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _steps(top, most):
    """(scale, reciprocal) of a maximum: each a quotient rounded to fp32 (by way
    of 64 bits: they decide ties)."""
    s = torch.where(top > 0, (top.double() / most).float().clamp(min=TINY), torch.ones_like(top))
    return s, (1.0 / s.double()).float()


def _int8_plain(x):
    x = x.float()
    s, inv = _steps(x.abs().amax(1), INT8_MAX)
    q = torch.round(x * inv[:, None]).clamp(-INT8_MAX, INT8_MAX)
    return q.to(torch.int8), s


def _fp8_plain(x):
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x, (0, _blocks(cols) * BLOCK - cols)).view(rows, -1, BLOCK)
    s, inv = _steps(pad.abs().amax(2), E4M3_MAX)
    q = (pad * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :cols]
    return q.to(torch.float8_e4m3fn), s


def _norm_plain(s):
    v, out = s["rows"].float(), []
    if s["residual"] is not None:
        r = (v + s["residual"].float()).to(s["residual"].dtype)
        v, out = r.float(), [r]
    # 64 bits: the codes go by the scale's last bit
    inv = (1.0 / torch.sqrt(v.double().square().sum(1) / v.shape[1] + EPS)).float()
    n = v * inv[:, None] * s["weight"].float()
    if s["y"]:
        out.append(n.to(TYPES[s["y"]]))
    if s["codes"]:
        out.extend(_int8_plain(n) if s["codes"] == "int8" else _fp8_plain(n))
    return out


def _linear_plain(x, xs, w, ws):
    if xs is None:
        x, xs = _int8_plain(x)
    return x.float() @ w.float().t() * xs[:, None] * ws


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        return _norm_plain(s)
    if s["op"] == "quantize":
        return _int8_plain(s["x"])
    if s["op"] == "linear":
        return _linear_plain(s["x"], s["xs"], s["w"], s["ws"]).to(TYPES[s["out"]])
    gate = _linear_plain(s["x"], s["xs"], *s["gate"])
    up = _linear_plain(s["x"], s["xs"], *s["up"])
    h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)
    return _linear_plain(h, None, *s["down"]).to(torch.bfloat16)


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _run_own(s):
    from nvfp4_routed_expert_amd import native
    if s["op"] == "norm":
        r = native.rms_norm_quantize(s["rows"], s["weight"], residual=s["residual"], eps=EPS,
                                     codes=s["codes"] or None,
                                     y_dtype=TYPES[s["y"]] if s["y"] else None)
        codes = r.codes.view(torch.float8_e4m3fn) if s["codes"] == "fp8" else r.codes
        return [t for t in (r.residual, r.y, codes, r.scales) if t is not None]
    if s["op"] == "quantize":
        return native.int8_quantize(s["x"])
    if s["op"] == "linear":
        return native.int8_linear(s["x"], s["w"], s["ws"], x_scales=s["xs"],
                                  out_dtype=TYPES[s["out"]])
    return native.int8_mlp(s["x"], s["gate"], s["up"], s["down"], x_scales=s["xs"])


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_scales(x, most):
    """Scale and reciprocal of the maxima of the last axis, which the quantisers
    define by 32-bit steps; formed in 64 bits and rounded."""
    top = np.abs(x).max(-1)
    s = np.where(top > 0, np.maximum(top / most, TINY), 1.0).astype(np.float32)
    return s, (1.0 / s.astype(np.float64)).astype(np.float32)


def _exact_int8(x):
    """Integers and scales (numpy) of fp32 values held in 64 bits."""
    s, inv = _exact_scales(x, INT8_MAX)
    v = (x * inv[:, None].astype(np.float64)).astype(np.float32)
    return np.clip(np.rint(v), -INT8_MAX, INT8_MAX), s


def _exact_fp8(x):
    q, s = np.empty_like(x), []
    for b in range(0, x.shape[1], BLOCK):
        sc, inv = _exact_scales(x[:, b:b + BLOCK], E4M3_MAX)
        v = (x[:, b:b + BLOCK] * inv[:, None].astype(np.float64)).astype(np.float32)
        a = np.minimum(np.abs(v.astype(np.float64)), E4M3_MAX)
        ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0) - 3.0)
        q[:, b:b + BLOCK] = np.copysign(np.rint(a / ulp) * ulp, v)
        s.append(sc)
    return q, np.stack(s, 1)


def _exact_norm(s, case):
    v, out = s["rows"].double(), []
    if s["residual"] is not None:
        # (sums of two bf16 or fp32 numbers: one rounding to fp32, one to the stream's type)
        r = (v + s["residual"].double()).float().to(s["residual"].dtype)
        v, out = r.double(), [v + s["residual"].double()]
    v, w = v.cpu().numpy(), s["weight"].double().cpu().numpy()
    inv = 1.0 / np.sqrt((v * v).mean(1) + EPS)
    if case["y"]:
        out.append(v * inv[:, None] * w)
    if case["codes"]:
        # the codes' 32-bit steps
        f = (v * inv.astype(np.float32)[:, None].astype(np.float64)).astype(np.float32)
        n = (f.astype(np.float64) * w).astype(np.float32).astype(np.float64)
        q, sc = _exact_int8(n) if case["codes"] == "int8" else _exact_fp8(n)
        out += [q.astype(np.int8) if case["codes"] == "int8" else q, sc.astype(np.float64)]
    return out


def _exact_product(x, xs, w, ws):
    """x: integers in 64 bits (their sums stay exact)."""
    return (x @ w.double().t()) * (xs.double()[:, None] * ws.double()[None, :])


def _exact_rows(x, xs):
    if xs is not None:
        return x.double(), xs
    q, s = _exact_int8(x.double().cpu().numpy())
    return torch.from_numpy(q).to(x.device).double(), torch.from_numpy(s).to(x.device)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "quantize":
        if case["rows"] * case["cols"] > 1 << 25:
            s["x"] = s["x"].double()
            top = s["x"].abs().amax(1)
            sc = torch.where(top > 0, (top / INT8_MAX).clamp(min=TINY), 1.0 + 0 * top).float()
            inv = (1.0 / sc.double()).float().double()
            q = torch.round((s["x"] * inv[:, None]).float().double())
            return q.clamp(-INT8_MAX, INT8_MAX).to(torch.int8), sc.double()
        q, sc = _exact_int8(s["x"].double().cpu().numpy())
        return q.astype(np.int8), sc.astype(np.float64)
    x, xs = _exact_rows(s["x"], s["xs"])
    if case["op"] == "linear":
        return _exact_product(x, xs, s["w"], s["ws"])
    gate, up = _exact_product(x, xs, *s["gate"]), _exact_product(x, xs, *s["up"])
    h = (gate * torch.special.expit(gate) * up).to(torch.bfloat16)
    return _exact_product(*_exact_rows(h, None), *s["down"])
