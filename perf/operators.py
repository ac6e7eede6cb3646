"""Measured cases of the FP8 block-scaled operators and of the one-call MoE layer.

Four operators, each in its plain form (elementary torch operations) and, with
`own` set, as a user calls the library:

  quantize  native.fp8_block_quantize   E4M3 codes and one fp32 scale per 1 x 128
                                        (activations) or 128 x 128 (weights) block
  linear    native.fp8_block_linear     y = x . W^T on such operands
  mlp       native.fp8_block_mlp        gated MLP with FP8 weights, x and h quantised
                                        online
  layer     native.moe_layer_decode     router, top-k, NVFP4 routed experts and BF16
                                        shared expert of a few tokens
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # a decode batch's activations in front of a projection (a latency-bound call)
        dict(name="quantize act 16x5120", op="quantize", rows=16, cols=5120, block=1, dtype="bf16"),
        # a checkpoint's fp32 MLP matrix turned into FP8 weights
        dict(name="quantize weight 17408x5120", op="quantize", rows=17408, cols=5120, block=128,
             dtype="f32"),
        # one token through the widest projection of a dense block
        dict(name="linear M1 17408x5120", op="linear", M=1, N=17408, K=5120, pre=False, out="bf16"),
        # a decode batch through a short projection (few rows, long K)
        dict(name="linear M8 5120x17408", op="linear", M=8, N=5120, K=17408, pre=False, out="bf16"),
        # a ragged batch: N no multiple of a tile, K with a partial last block, fp32 out
        dict(name="linear M77 5000x2080", op="linear", M=77, N=5000, K=2080, pre=False, out="f32"),
        # a prefill chunk on operands quantised once for several projections
        dict(name="linear M2048 17408x5120", op="linear", M=2048, N=17408, K=5120, pre=True,
             out="bf16"),
        # one token through a dense FP8 MLP block
        dict(name="mlp T1 5120x17408", op="mlp", T=1, H=5120, I=17408),
        # a small batch, intermediate size with a partial last block
        dict(name="mlp T24 2048x1056", op="mlp", T=24, H=2048, I=1056),
        # a prefill chunk through a dense FP8 MLP block
        dict(name="mlp T512 5120x17408", op="mlp", T=512, H=5120, I=17408),
        # one user's decode step of a 512-expert layer with a gated shared expert
        dict(name="layer T1 E512", op="layer", T=1, H=2048, I=512, E=512, k=8, Is=512, gate=True,
             renorm=True, bias=False),
        # a decode batch of the same layer
        dict(name="layer T16 E512", op="layer", T=16, H=2048, I=512, E=512, k=8, Is=512, gate=False,
             renorm=True, bias=False),
        # a larger batch of a layer with fewer, wider experts and no shared expert
        dict(name="layer T32 E128", op="layer", T=32, H=4096, I=1536, E=128, k=8, Is=0, gate=False,
             renorm=False, bias=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "mlp", "layer", "layer"])
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, 16384), cols=_log_int(rng, 32, 8192, 32),
                    block=rng.choice([1, 1, 128]), dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 2048), N=_log_int(rng, 17, 17408),
                    K=_log_int(rng, 32, 5120, 32), pre=rng.random() < 0.5,
                    out=rng.choice(["bf16", "f32"]))
    if op == "mlp":
        return dict(op=op, T=_log_int(rng, 1, 512), H=_log_int(rng, 256, 5120, 32),
                    I=_log_int(rng, 96, 17408, 32))
    E = _log_int(rng, 8, 512)
    k = rng.randint(1, min(E, 10))
    T = min(_log_int(rng, 1, 64), 512 // k)
    H, I = _log_int(rng, 256, 4096, 32), _log_int(rng, 96, 1536, 32)
    E = max(k, min(E, 128 * 4096 * 1536 // (H * I)))
    Is = rng.choice([0, I, _log_int(rng, 96, 2048, 32)])
    return dict(op=op, T=T, H=H, I=I, E=E, k=k, Is=Is, gate=Is > 0 and rng.random() < 0.5,
                renorm=rng.random() < 0.7, bias=rng.random() < 0.3)


def _blocks(n):
    return -(-n // BLOCK)


def work(c):
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        sc = (c["rows"] if c["block"] == 1 else _blocks(c["rows"])) * _blocks(c["cols"])
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + n + 4 * sc, "flops": 2 * n}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        x = M * K + 4 * M * _blocks(K) if c["pre"] else 2 * M * K
        w = N * K + 4 * _blocks(N) * _blocks(K)
        return {"bytes": x + w + M * N * (2 if c["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    if c["op"] == "mlp":
        T, H, I = c["T"], c["H"], c["I"]
        w = 3 * (H * I + 4 * _blocks(H) * _blocks(I))
        return {"bytes": w + 4 * T * H, "flops": 6 * T * H * I}
    T, H, I, E, k, Is = (c[n] for n in ("T", "H", "I", "E", "k", "Is"))
    active = E * (1.0 - (1.0 - k / E) ** T)       # expected distinct experts of the batch
    w = active * 3 * H * I * 9 / 16 + 2 * E * H + 6 * H * Is
    return {"bytes": w + 4 * T * H + 8 * T * k,
            "flops": 6 * T * k * H * I + 2 * T * E * H + 6 * T * H * Is}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _acts(g, rows, cols):
    """Activations with channels of different strength, as in front of a projection."""
    strength = torch.exp(0.5 * _randn(g, 1, cols))
    return _randn(g, rows, cols) * strength


def _fp8_weight(g, n, k):
    """codes uint8 [n, k] and scales f32 [ceil(n/128), ceil(k/128)] of N(0, 0.02) weights."""
    q, s = _quantize_plain(_randn(g, n, k, std=0.02), BLOCK)
    return q.view(torch.uint8), s


def _nvfp4_weight(g, e, n, k):
    """e stacked NVFP4 matrices [n, k] of N(0, 0.02) weights: codes, scales, globals."""
    codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((e, n, k // 16), dtype=torch.uint8, device="cuda")
    glob = torch.empty(e, dtype=torch.float32, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // (n * k))
    for a in range(0, e, step):
        b = min(e, a + step)
        w = _randn(g, b - a, n, k // 16, 16, std=0.02)
        top = w.abs().amax(-1)
        gl = top.amax((1, 2)) / 2688.0
        s = (top / (6.0 * gl[:, None, None])).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
        unit = s.float() * gl[:, None, None]
        v = w / torch.where(unit > 0, unit, torch.ones_like(unit))[..., None]
        c = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8)
        c |= (v < 0).to(torch.uint8) << 3
        c = c.view(b - a, n, k // 2, 2)
        codes[a:b] = c[..., 0] | (c[..., 1] << 4)
        scales[a:b] = s.view(torch.uint8)
        glob[a:b] = gl
    return codes, scales, glob


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quantize":
        weight = case["block"] == BLOCK
        x = _randn(g, case["rows"], case["cols"], std=0.02) if weight else \
            _acts(g, case["rows"], case["cols"])
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
    elif case["op"] == "linear":
        x = _acts(g, case["M"], case["K"]).to(torch.bfloat16)
        s["w"], s["ws"] = _fp8_weight(g, case["N"], case["K"])
        if case["pre"]:
            q, s["xs"] = _quantize_plain(x.float(), 1)
            s["x"] = q.view(torch.uint8)
        else:
            s["x"], s["xs"] = x, None
    elif case["op"] == "mlp":
        s["x"] = _acts(g, case["T"], case["H"]).to(torch.bfloat16)
        for name, n, k in (("gate", case["I"], case["H"]), ("up", case["I"], case["H"]),
                           ("down", case["H"], case["I"])):
            s[name], s[name + "_s"] = _fp8_weight(g, n, k)
    else:
        T, H, I, E, Is = (case[n] for n in ("T", "H", "I", "E", "Is"))
        bf = torch.bfloat16
        s["x"] = _randn(g, T, H).to(bf)
        s["router"] = _randn(g, E, H, std=H ** -0.5).to(bf)
        s["rbias"] = _randn(g, E, std=0.5) if case["bias"] else None
        for name, n, k in (("gate", I, H), ("up", I, H), ("down", H, I)):
            s[name], s[name + "_s"], s[name + "_g"] = _nvfp4_weight(g, E, n, k)
        s["shared"] = tuple(_randn(g, *d, std=0.02).to(bf)
                            for d in ((Is, H), (Is, H), (H, Is))) if Is else None
        s["sgate"] = _randn(g, H, std=H ** -0.5).to(bf) if case["gate"] else None
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _quantize_plain(x, block):
    """(codes float8_e4m3fn [R, C], scales f32): every step one operation rounded
    to fp32 (the quotients by way of 64 bits: they decide ties)."""
    r, c = x.shape
    cb = _blocks(c)
    rb = r if block == 1 else _blocks(r)
    pad = torch.nn.functional.pad(x.float(), (0, cb * BLOCK - c, 0, rb * block - r))
    pad = pad.view(rb, block, cb, BLOCK)
    top = pad.abs().amax((1, 3))
    s = torch.where(top > 0, (top.double() / E4M3_MAX).float().clamp(min=TINY),
                    torch.ones_like(top))
    v = pad * (1.0 / s.double()).float()[:, None, :, None]
    q = v.clamp(-E4M3_MAX, E4M3_MAX).view(rb * block, cb * BLOCK)[:r, :c]
    return q.to(torch.float8_e4m3fn), s


def _spread(scales, rows, cols, block):
    """Block scales as one scale per element, [rows, cols]."""
    s = scales.repeat_interleave(BLOCK, 1)[:, :cols]
    return s if block == 1 else s.repeat_interleave(block, 0)[:rows]


def _fp8_values(codes, scales, block):
    return codes.view(torch.float8_e4m3fn).float() * _spread(scales, *codes.shape, block)


def _linear_plain(x, xs, w, ws):
    if xs is None:
        x, xs = _quantize_plain(x, 1)
    return _fp8_values(x, xs, 1) @ _fp8_values(w, ws, BLOCK).t()


def _silu_mul(a, b):
    return a / (1.0 + torch.exp(-a)) * b


def _nvfp4_values(codes, scales, glob, ids):
    """fp32 values [P, n, k] of the experts ids."""
    c = codes[ids]
    both = torch.stack((c & 15, c >> 4), -1).flatten(-2).int()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[both].unflatten(-1, (-1, 16))
    v = v * scales[ids].view(torch.float8_e4m3fn).float()[..., None]
    return v.flatten(-2) * glob[ids][:, None, None]


def _layer_plain(s):
    T, k = s["T"], s["k"]
    x = s["x"].float()
    # 64 bits: a near tie between two experts must not be decided by the sum's order
    logits = (s["x"].double() @ s["router"].double().t()).float()
    if s["rbias"] is not None:
        logits = logits + s["rbias"]
    vals, order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = order[:, :k]
    e = torch.exp(vals - vals[:, :1])
    wts = e[:, :k] / (e[:, :k] if s["renorm"] else e).sum(1, keepdim=True)
    flat = ids.reshape(-1)
    xp = x.repeat_interleave(k, 0)[:, :, None]
    gate = torch.bmm(_nvfp4_values(s["gate"], s["gate_s"], s["gate_g"], flat), xp)[..., 0]
    up = torch.bmm(_nvfp4_values(s["up"], s["up_s"], s["up_g"], flat), xp)[..., 0]
    h = _silu_mul(gate, up).to(torch.bfloat16).float()
    down = torch.bmm(_nvfp4_values(s["down"], s["down_s"], s["down_g"], flat), h[..., None])[..., 0]
    y = (down.view(T, k, -1) * wts[..., None]).sum(1)
    if s["shared"] is not None:
        wg, wu, wd = (w.float() for w in s["shared"])
        sh = _silu_mul(x @ wg.t(), x @ wu.t()).to(torch.bfloat16).float() @ wd.t()
        if s["sgate"] is not None:
            sh = sh / (1.0 + torch.exp(-(x @ s["sgate"].float())))[:, None]
        y = y + sh
    return y.to(torch.bfloat16), ids.int(), wts


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "quantize":
        return _quantize_plain(s["x"], s["block"])
    if s["op"] == "linear":
        y = _linear_plain(s["x"], s["xs"], s["w"], s["ws"])
        return y if s["out"] == "f32" else y.to(torch.bfloat16)
    if s["op"] == "mlp":
        gate = _linear_plain(s["x"], None, s["gate"], s["gate_s"])
        up = _linear_plain(s["x"], None, s["up"], s["up_s"])
        h = _silu_mul(gate, up).to(torch.bfloat16)
        return _linear_plain(h, None, s["down"], s["down_s"]).to(torch.bfloat16)
    return _layer_plain(s)


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _run_own(s):
    from nvfp4_routed_expert_amd import native
    if s["op"] == "quantize":
        codes, scales = native.fp8_block_quantize(s["x"], block_rows=s["block"])
        return codes.view(torch.float8_e4m3fn), scales
    if s["op"] == "linear":
        return native.fp8_block_linear(s["x"], s["w"], s["ws"], x_scales=s["xs"],
                                       out_dtype=torch.float32 if s["out"] == "f32"
                                       else torch.bfloat16)
    if s["op"] == "mlp":
        return native.fp8_block_mlp(s["x"], (s["gate"], s["gate_s"]), (s["up"], s["up_s"]),
                                    (s["down"], s["down_s"]))
    weights = native.ExpertWeights(s["gate"], s["gate_s"], s["gate_g"], s["up"], s["up_s"],
                                   s["up_g"], s["down"], s["down_s"], s["down_g"])
    y, (ids, wts) = native.moe_layer_decode(s["x"], s["router"], weights, s["k"],
                                            renormalize=s["renorm"], bias=s["rbias"],
                                            shared=s["shared"], shared_gate=s["sgate"])
    return y, ids, wts


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _e4m3_grid(v):
    """Nearest E4M3 value of v (64 bits), ties to even, saturating."""
    a = v.abs().clamp(max=E4M3_MAX)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -30))).clamp(min=-6.0)
    ulp = torch.exp2(e - 3.0)
    return torch.copysign(torch.round(a / ulp) * ulp, v)


def _exact_quant(x, block):
    """(grid values, scales) per block.  The quantiser is defined by its 32-bit
    steps s = amax / 448, 1 / s and x * (1 / s): quotients of bf16 numbers by
    amax / 448 often lie on a tie, which those roundings decide.  Each step is
    formed in 64 bits (the product exactly) and rounded to 32."""
    x = x.double()
    q, s = torch.empty_like(x), []
    for b in range(0, x.shape[1], BLOCK):
        cols = x[:, b:b + BLOCK]
        top = cols.abs().amax(1)
        if block != 1:
            fill = torch.zeros(_blocks(len(top)) * block, dtype=top.dtype, device=top.device)
            fill[:len(top)] = top
            top = fill.view(-1, block).amax(1)
        sc = torch.where(top > 0, (top / E4M3_MAX).clamp(min=TINY), 1.0 + 0 * top).float()
        s.append(sc)
        inv = (1.0 / sc.double()).float().double()
        inv = inv if block == 1 else inv.repeat_interleave(block)[:x.shape[0]]
        q[:, b:b + BLOCK] = _e4m3_grid((cols * inv[:, None]).float().double())
    return q, torch.stack(s, 1)


def _exact_bytes(codes):
    """E4M3 bytes decoded through a table of all 256."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    mag = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    t = torch.from_numpy(np.where(b & 128, -mag, mag)).to(codes.device)
    return t[codes.int()]


def _exact_product(xq, xs, w, ws):
    y = 0.0
    for j, b in enumerate(range(0, xq.shape[1], BLOCK)):
        wb = _exact_bytes(w[:, b:b + BLOCK])
        row_scale = ws[:, j].double()[torch.arange(w.shape[0], device=w.device) // BLOCK]
        y = y + (xq[:, b:b + BLOCK] * xs[:, j:j + 1].double()) @ (wb * row_scale[:, None]).t()
    return y


def _sigmoid64(v):
    return torch.special.expit(v)


def _exact_expert(s, e, xt):
    def mat(name):
        c = s[name][e]
        n, half = c.shape
        v = torch.empty((n, 2 * half), dtype=torch.float64, device=c.device)
        t = torch.tensor(E2M1 + tuple(-u for u in E2M1), dtype=torch.float64, device=c.device)
        v[:, 0::2], v[:, 1::2] = t[(c & 15).int()], t[(c >> 4).int()]
        sc = _exact_bytes(s[name + "_s"][e])
        return v * sc.repeat_interleave(16, 1) * s[name + "_g"][e].double()
    gate, up = xt @ mat("gate").t(), xt @ mat("up").t()
    return (gate * _sigmoid64(gate) * up).to(torch.bfloat16).double() @ mat("down").t()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        q, sc = _exact_quant(s["x"], case["block"])
        return q, sc.double()
    if case["op"] == "linear":
        xq, xs = _exact_quant(s["x"], 1) if s["xs"] is None else (_exact_bytes(s["x"]), s["xs"])
        return _exact_product(xq, xs, s["w"], s["ws"])
    if case["op"] == "mlp":
        xq, xs = _exact_quant(s["x"], 1)
        gate = _exact_product(xq, xs, s["gate"], s["gate_s"])
        up = _exact_product(xq, xs, s["up"], s["up_s"])
        h = (gate * _sigmoid64(gate) * up).to(torch.bfloat16)
        return _exact_product(*_exact_quant(h, 1), s["down"], s["down_s"])
    x = s["x"].double()
    logits = x @ s["router"].double().t()
    if s["rbias"] is not None:
        logits = logits + s["rbias"].double()
    order = torch.argsort(-logits, dim=1, stable=True)[:, :case["k"]]
    picked = logits.gather(1, order)
    den = torch.logsumexp(picked if case["renorm"] else logits, 1, keepdim=True)
    wts = torch.exp(picked - den)
    y = torch.zeros_like(x)
    for e in order.unique().tolist():
        t, j = (order == e).nonzero(as_tuple=True)
        y.index_add_(0, t, _exact_expert(s, e, x[t]) * wts[t, j][:, None])
    if s["shared"] is not None:
        wg, wu, wd = (w.double() for w in s["shared"])
        g = x @ wg.t()
        sh = (g * _sigmoid64(g) * (x @ wu.t())).to(torch.bfloat16).double() @ wd.t()
        if s["sgate"] is not None:
            sh = sh * _sigmoid64(x @ s["sgate"].double())[:, None]
        y = y + sh
    return y, None, wts
