"""moe_layer_decode (a whole MoE layer for a few tokens) against a plain 64-bit
form, against the separate calls, and in the ways a decode loop uses it."""
import sys

import numpy as np
import pytest
import torch

from helpers import assert_bf16_output, assert_close_f32
from nvfp4_routed_expert_amd import native

pytestmark = pytest.mark.gpu
DEV = "cuda"
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def nvfp4_stack(e, n, k, seed):
    """e stacked NVFP4 matrices (device) from N(0, 0.02) weights."""
    g = torch.Generator().manual_seed(seed)
    out = [], [], []
    for _ in range(e):
        w = torch.randn(n, k, generator=g) * 0.02
        for lst, t in zip(out, native.nvfp4_quantize(w.to(DEV))):
            lst.append(t)
    c, s, gl = out
    return torch.stack(c), torch.stack(s), torch.cat(gl)


def e4m3(b):
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    return np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)


def nvfp4_values(codes, scales, g, e):
    c = codes[e].cpu().numpy()
    v = np.stack([E2M1[c & 15], E2M1[c >> 4]], -1).reshape(c.shape[0], -1)
    return v * np.repeat(e4m3(scales[e].cpu().numpy()), 16, 1) * float(g[e])


class Layer:
    def __init__(self, T, H, I, E, k, Is=0, gate=False, bias=False, seed=0, twins=False):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.x = rn(T, H).to(torch.bfloat16).to(DEV)
        r = (rn(E, H) * H ** -0.5).to(torch.bfloat16)
        if twins:
            r[1::2] = r[0:E - 1:2][: r[1::2].shape[0]]
        self.router = r.to(DEV)
        self.bias = (rn(E) * 0.5).to(DEV) if bias else None
        mats = [nvfp4_stack(E, I, H, seed + 1), nvfp4_stack(E, I, H, seed + 2),
                nvfp4_stack(E, H, I, seed + 3)]
        self.w = native.ExpertWeights(*mats[0], *mats[1], *mats[2])
        self.mats = mats
        self.shared = tuple((rn(*d) * 0.02).to(torch.bfloat16).to(DEV)
                            for d in ((Is, H), (Is, H), (H, Is))) if Is else None
        self.sgate = (rn(H) * H ** -0.5).to(torch.bfloat16).to(DEV) if gate else None
        self.Is = Is

    def workspace(self, T=None):
        n = native.lib().moe_layer_decode_workspace_size(T or self.T, self.H, self.I, self.E,
                                                         self.k, self.Is)
        return torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xA5)   # any contents will do

    def run(self, **kw):
        kw.setdefault("x", self.x)
        x = kw.pop("x")
        return native.moe_layer_decode(x, self.router, self.w, self.k, bias=self.bias,
                                       shared=self.shared, shared_gate=self.sgate, **kw)

    def ref(self, renorm=True, x=None):
        x = (self.x if x is None else x).double().cpu().numpy()
        logits = x @ self.router.double().cpu().numpy().T
        if self.bias is not None:
            logits = logits + self.bias.double().cpu().numpy()
        order = np.argsort(-logits, axis=1, kind="stable")
        ids = order[:, :self.k]
        srt = np.take_along_axis(logits, order, 1)
        gaps = (srt[:, :-1] - srt[:, 1:])[:, :self.k]
        ex = np.exp(srt - srt[:, :1])
        wts = ex[:, :self.k] / (ex[:, :self.k] if renorm else ex).sum(1, keepdims=True)
        y = np.zeros_like(x)
        silu_mul = lambda a, b: bf16(a / (1 + np.exp(-a)) * b)
        for e in np.unique(ids):
            t, j = np.nonzero(ids == e)
            gw, uw, dw = (nvfp4_values(*m, e) for m in self.mats)
            y[t] += (silu_mul(x[t] @ gw.T, x[t] @ uw.T) @ dw.T) * wts[t, j][:, None]
        if self.shared is not None:
            wg, wu, wd = (w.double().cpu().numpy() for w in self.shared)
            s = silu_mul(x @ wg.T, x @ wu.T) @ wd.T
            if self.sgate is not None:
                s = s / (1 + np.exp(-(x @ self.sgate.double().cpu().numpy())))[:, None]
            y = y + s
        return y, ids, wts, gaps


def bf16(v):
    return torch.from_numpy(np.asarray(v)).to(torch.bfloat16).double().numpy()


def clear_gaps(ids, gaps):
    """Tokens whose choice and order no fp32 sum can change (logit sums of
    unit-variance products: far below 1e-5 apart)."""
    return (gaps > 1e-5).all(1)


#        T   H     I     E     k   Is   gate   bias   renorm
CASES = [(1, 256, 128, 8, 2, 0, False, False, True),
         (1, 2048, 512, 16, 8, 512, True, False, True),
         (2, 4096, 1536, 4, 2, 0, False, False, True),
         (3, 320, 96, 5, 5, 64, False, True, False),
         (4, 4160, 64, 6, 1, 544, True, True, True),
         (5, 1056, 1056, 9, 3, 160, True, True, True),
         (6, 32, 32, 3, 2, 32, True, False, True),
         (7, 2080, 288, 40, 32, 96, False, False, False),
         (16, 2048, 512, 32, 8, 512, False, False, True),
         (33, 512, 2080, 6, 2, 2080, True, False, True),
         (51, 352, 224, 1024, 10, 0, False, False, True),
         (64, 256, 64, 1, 1, 32, False, False, True),
         (64, 512, 256, 16, 8, 256, False, False, True)]


@pytest.mark.parametrize("T,H,I,E,k,Is,gate,bias,renorm", CASES)
def test_layer(T, H, I, E, k, Is, gate, bias, renorm):
    say("layer", T, H, I, E, k, Is, gate, bias, renorm)
    L = Layer(T, H, I, E, k, Is, gate, bias, seed=T + H)
    ref, ids, wts, gaps = L.ref(renorm)
    y32, (gids, gw) = L.run(renormalize=renorm, out_dtype=torch.float32)
    ok = clear_gaps(ids, gaps)
    assert ok.mean() > 0.9
    assert np.array_equal(gids.cpu().numpy()[ok], ids[ok])
    np.testing.assert_allclose(gw.cpu().numpy()[ok], wts[ok], rtol=1e-5)
    assert_close_f32(y32.cpu().numpy()[ok], ref[ok], f"layer {T} {H} {I} {E} {k}")
    y16, (gids2, gw2) = L.run(renormalize=renorm)
    assert torch.equal(gids, gids2) and torch.equal(gw, gw2)
    assert_bf16_output(y16.float().cpu().numpy()[ok], y32.cpu().numpy()[ok], ref[ok], "layer bf16")


def test_ties_go_to_the_lower_expert():
    """Router rows in equal pairs: equal logits, the lower index first."""
    say("ties")
    L = Layer(9, 256, 64, 32, 6, seed=4, twins=True)
    _, ids, _, _ = L.ref()
    _, (gids, gw) = L.run()
    g = gids.cpu().numpy()
    assert np.array_equal(g, ids)
    assert np.all(g[:, 1::2] == g[:, 0::2] + 1)
    assert torch.equal(gw[:, 0::2], gw[:, 1::2])


def test_agrees_with_the_separate_calls():
    """moe_router_topk, moe_grouped_nvfp4_ffn and moe_shared_expert_ffn on the
    same inputs: the same experts, and outputs of the same sums."""
    T, H, I, E, k, Is = 12, 2048, 512, 64, 8, 512
    say("separate calls")
    L = Layer(T, H, I, E, k, Is, seed=8)
    ids, w, off, pairs, _ = native.moe_router_topk(L.x, L.router, k)
    y, _ = native.moe_grouped_nvfp4_ffn(L.x, L.w, ids, w, off, pairs, k, out_dtype=torch.float32)
    native.moe_shared_expert_ffn(L.x, *L.shared, y=y, accumulate=True)
    got, (gids, gw) = L.run(out_dtype=torch.float32)
    assert torch.equal(gids, ids)
    np.testing.assert_allclose(gw.cpu().numpy(), w.cpu().numpy(), rtol=1e-5)
    assert_close_f32(got.cpu().numpy(), y.double().cpu().numpy(), "separate calls")


def test_repeated_calls_on_one_workspace():
    """One workspace, larger and smaller batches in turn, each bit-identical to
    a call on a fresh workspace; outputs behind the batch are left alone."""
    say("workspace reuse")
    L = Layer(16, 512, 256, 24, 4, 128, gate=True, seed=3)
    ws = L.workspace()
    for T in (16, 1, 5, 16, 2, 2, 9):
        x = L.x[:T].contiguous()
        out = torch.full((18, 512), 3.0, dtype=torch.float32, device=DEV)
        y, (i, w) = L.run(x=x, workspace=ws, out=out[1:1 + T])
        y2, (i2, w2) = L.run(x=x, out_dtype=torch.float32)
        assert torch.equal(y, y2) and torch.equal(i, i2) and torch.equal(w, w2)
        assert torch.all(out[0] == 3.0) and torch.all(out[1 + T:] == 3.0)


def test_empty_batch():
    say("empty")
    L = Layer(1, 256, 64, 4, 2)
    y, (i, w) = L.run(x=L.x[:0].contiguous())
    assert y.shape == (0, 256) and i.shape == (0, 2)


def test_graph_replays():
    """Two captured graphs (a workspace each) replayed in turn with eager calls
    between: every replay equals the eager result."""
    say("graph")
    L = Layer(8, 512, 256, 32, 4, 128, gate=True, seed=6)
    graphs = []
    for T in (8, 3):
        x = L.x[:T].contiguous()
        ws = L.workspace(T)
        y = torch.empty((T, 512), dtype=torch.float32, device=DEV)
        route = (torch.empty((T, 4), dtype=torch.int32, device=DEV),
                 torch.empty((T, 4), dtype=torch.float32, device=DEV))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.run(x=x, workspace=ws, out=y, route_out=route)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.run(x=x, workspace=ws, out=y, route_out=route)
        graphs.append((g, x, y, route, ws))          # (the graph needs its workspace)
    for seed in range(4):
        for g, x, y, route, _ in graphs:
            gen = torch.Generator().manual_seed(100 + seed)
            x.copy_(torch.randn(x.shape, generator=gen).to(torch.bfloat16))
            want, (i, w) = L.run(x=x, out_dtype=torch.float32)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(route[0], i) and torch.equal(route[1], w)


def test_two_streams_at_once():
    """Calls on two streams with a workspace each, queued without waiting: the
    items of one wait only for their own launch's, so both finish."""
    say("two streams")
    L = Layer(16, 1024, 512, 64, 8, 256, seed=7)
    M = Layer(4, 1024, 512, 64, 8, 256, seed=9)
    want = [a.run(out_dtype=torch.float32)[0] for a in (L, M)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [a.workspace() for a in (L, M)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(6):
        for n, a in enumerate((L, M)):
            with torch.cuda.stream(streams[n]):
                outs[n].append(a.run(workspace=spaces[n], out_dtype=torch.float32)[0])
    torch.cuda.synchronize()
    for n in range(2):
        for y in outs[n]:
            assert torch.equal(y, want[n])


def test_decode_block_with_fp8_projections():
    """The operators as a mixed checkpoint's decoder block uses them: an FP8
    projection in front of the MoE layer, its output through a dense FP8 MLP,
    against the same chain of separately checked steps on the host."""
    say("block")
    T, H = 6, 512
    L = Layer(T, H, 256, 16, 4, 128, gate=True, seed=12)
    g = torch.Generator().manual_seed(5)
    ws = [native.fp8_block_quantize((torch.randn(*s, generator=g) * 0.05).to(DEV), 128)
          for s in ((H, H), (640, H), (640, H), (H, 640))]
    x0 = L.x
    a = native.fp8_block_linear(x0, *ws[0])
    y, _ = L.run(x=a)
    z = native.fp8_block_mlp(y, *ws[1:])
    # each step from the previous step's device output
    ref, _, _, gaps = L.ref(x=a)
    ok = (gaps > 1e-5).all(1)
    rel = np.linalg.norm(y.double().cpu().numpy()[ok] - ref[ok]) / np.linalg.norm(ref[ok])
    assert rel <= 2.0 ** -8          # one bf16 rounding, at most 2^-8 relative
    codes, s = native.fp8_block_quantize(x0)
    assert torch.equal(a, native.fp8_block_linear(codes, *ws[0], x_scales=s))
    assert torch.isfinite(z.float()).all() and z.shape == (T, H)


@pytest.mark.parametrize("T,H,I,E,k,Is,gate,bias,renorm",
                         [(9, 8192, 160, 3, 2, 0, False, False, True),
                          (12, 4096, 288, 3, 2, 64, True, False, True),
                          (12, 4128, 288, 3, 2, 64, True, False, True),
                          (5, 544, 512, 4, 2, 0, False, True, True),
                          (64, 1024, 1024, 2, 1, 0, False, False, True)])
def test_layer_of_crowded_experts(T, H, I, E, k, Is, gate, bias, renorm):
    """Several segments per expert, of up to four tokens or (H > 4096) two."""
    test_layer(T, H, I, E, k, Is, gate, bias, renorm)


@pytest.mark.parametrize("T,H,I,E,k,Is,gate,bias,renorm",
                         [(1, 4160, 2336, 8, 8, 0, False, False, True),
                          (20, 8192, 288, 4, 4, 0, False, False, True),
                          (33, 2080, 1056, 8, 8, 32, True, False, True)])
def test_layer_of_large_experts(T, H, I, E, k, Is, gate, bias, renorm):
    """Codes past the size from which they are loaded as used once.  The bf16
    outputs are the f32 ones rounded, element by element.  (Their Frobenius
    distance to the rounded oracle is no bound of its own: an f32 deviation d,
    here the roundings of h that fall the other way, moves a fraction d / u of
    the elements by a step u, sqrt(d u) together; d = 3e-4, a third of the f32
    limit, and u = 2^-7.5 give 1.3e-3.)"""
    say("layer", T, H, I, E, k, Is, gate, bias, renorm)
    L = Layer(T, H, I, E, k, Is, gate, bias, seed=T + H)
    ref, ids, wts, gaps = L.ref(renorm)
    y32, (gids, gw) = L.run(renormalize=renorm, out_dtype=torch.float32)
    ok = clear_gaps(ids, gaps)
    assert ok.mean() > 0.9
    assert np.array_equal(gids.cpu().numpy()[ok], ids[ok])
    np.testing.assert_allclose(gw.cpu().numpy()[ok], wts[ok], rtol=1e-5)
    print("rel_frob, max/rms:", assert_close_f32(y32.cpu().numpy()[ok], ref[ok], "large experts"),
          flush=True)
    y16, _ = L.run(renormalize=renorm)
    assert torch.equal(y16, y32.to(torch.bfloat16))


@pytest.mark.parametrize("E,k", [(5, 5), (40, 6), (600, 8)])
def test_logits_of_any_bits_choose_valid_experts(E, k):
    """Biases that turn every logit into the NaN of all one bits (the lowest
    order key): k different experts all the same, since ids address weights.
    The values are unspecified."""
    say("nan logits", E, k)
    L = Layer(3, 256, 32, E, k, seed=2, bias=True)
    L.bias.view(torch.int32).fill_(-1)
    y, (ids, _) = L.run()
    torch.cuda.synchronize()
    for row in ids.tolist():
        assert len(set(row)) == k and min(row) >= 0 and max(row) < E
    # one expert alone: it ranks last
    L.bias.zero_()
    L.bias.view(torch.int32)[1] = -1
    _, (ids, _) = L.run()
    torch.cuda.synchronize()
    for row in ids.tolist():
        assert len(set(row)) == k and min(row) >= 0 and max(row) < E
        assert (1 in row) == (k == E) and (k < E or row[-1] == 1)


def test_workspace_of_the_largest_batch():
    """One workspace of the size of 16 tokens (slices of 256 columns) for fewer
    (of 128, with more partial rows), each as on a workspace of its own."""
    say("workspace of the largest batch")
    L = Layer(16, 256, 512, 24, 8, 32, gate=True, seed=14)
    ws = L.workspace()
    for T in (16, 15, 3, 16, 14, 1):
        x = L.x[:T].contiguous()
        y, (i, w) = L.run(x=x, workspace=ws, out_dtype=torch.float32)
        y2, (i2, w2) = L.run(x=x, workspace=L.workspace(T), out_dtype=torch.float32)
        assert torch.equal(y, y2) and torch.equal(i, i2) and torch.equal(w, w2)


# ---- every compiled kernel ---------------------------------------------------------

# A case for each kernel that CASES and the tests above leave out: (T, H, I, E, k,
# Is, gate, bias, renorm) and what it takes: columns of a slice, H and I multiples
# of 128, tokens of a pass over an expert's weights, codes loaded as used once.
KERNEL_CASES = [((5, 512, 256, 5, 2, 0, False, False, True), (128, True, 4, False)),
                ((1, 320, 96, 5, 5, 32, True, False, True), (128, False, 1, False)),
                ((1, 4096, 2432, 8, 8, 0, False, False, True), (128, True, 1, True)),
                ((2, 4096, 1280, 16, 8, 0, False, True, True), (128, True, 2, True)),
                ((15, 1280, 512, 8, 8, 0, False, False, False), (128, True, 4, True)),
                ((15, 1376, 480, 8, 8, 96, False, False, True), (128, False, 4, True)),
                ((1, 256, 2048, 32, 32, 64, False, False, True), (256, True, 1, False)),
                ((1, 288, 2080, 32, 32, 0, False, False, True), (256, False, 1, False)),
                ((1, 1280, 8192, 8, 8, 0, False, False, True), (256, True, 1, True)),
                ((1, 1312, 8224, 8, 8, 0, False, True, True), (256, False, 1, True)),
                ((16, 256, 512, 256, 8, 512, True, False, True), (256, True, 2, False)),
                ((2, 1312, 1056, 33, 32, 0, False, False, False), (256, False, 2, True)),
                ((16, 1280, 512, 256, 8, 0, False, False, True), (256, True, 2, True))]


@pytest.mark.parametrize("case,plan", KERNEL_CASES)
def test_every_kernel(case, plan):
    T, H, I, E, k = case[:5]
    cols, tokens, once = native.layer_debug_plan(T, H, I, E, k)
    assert (cols, H % 128 == 0 and I % 128 == 0, tokens, once) == plan
    test_layer_of_large_experts(*case)


# ---- activations of very different magnitude ---------------------------------------


def integer_stack(e, n, k, seed, clear_first):
    """e NVFP4 matrices of random codes, block scales 0.5, 1 or 2 and global
    scale 2^-4: sums of their products with small integers times a power of two
    are exact in fp32.  clear_first: column 0 is zero."""
    r = np.random.default_rng(seed)
    codes = r.integers(0, 256, (e, n, k // 2), np.uint8)
    if clear_first:
        codes[:, :, 0] &= 0xF0
    scales = r.choice(np.array([0x30, 0x38, 0x40], np.uint8), (e, n, k // 16))
    put = lambda a: torch.from_numpy(a).to(DEV)
    return put(codes), put(scales), torch.full((e,), 2.0 ** -4, device=DEV)


@pytest.mark.parametrize("T,H,I,E,k", [(9, 320, 96, 1, 1), (10, 1056, 288, 2, 2),
                                       (2, 4128, 128, 2, 1), (6, 512, 256, 3, 2)])
def test_tokens_of_different_magnitudes(T, H, I, E, k):
    """x is used as two pieces by way of a power of two per token, h of one per
    token and slice.  Tokens from 2^-20 to 2^20 in one segment, one that is all
    zero, and one whose channel 0 is 2^20 times the rest (with zero weights in
    that channel: the rest, at the bottom of the pieces' range, must count in
    full).  x is small integers, gate and up are exact, so h is known up to expf;
    the down sums may be off by the pieces' 2^-21 of the largest h, 2^-12 of a
    block's largest product (16 products aligned to it with about 17 bits, twice
    for the two pieces) and the roundings of fp32.  Row by row."""
    say("magnitudes", T, H, I, E, k)
    r = np.random.default_rng(T)
    exps = np.array([0, -20, 20, 7, 0, -9, 14, 0, 3, -14])[:T]
    base = r.integers(-3, 4, (T, H)).astype(np.float64)
    base[:, 1] = 3.0
    base[min(7, T - 1)] = 0.0
    x = base * 2.0 ** exps[:, None]
    outlier = 4 if T > 4 else 0
    x[outlier, 0] = 2.0 ** 20
    L = Layer(T, H, I, E, k, seed=3)
    L.mats = [integer_stack(E, I, H, 1, True), integer_stack(E, I, H, 2, True),
              integer_stack(E, H, I, 3, False)]
    L.w = native.ExpertWeights(*L.mats[0], *L.mats[1], *L.mats[2])
    y, (ids, wts) = L.run(x=torch.from_numpy(x).to(torch.bfloat16).to(DEV), out_dtype=torch.float32)
    y, ids, wts = y.double().cpu().numpy(), ids.cpu().numpy(), wts.double().cpu().numpy()
    ref, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        gw, uw, dw = (nvfp4_values(*m, e) for m in L.mats)
        g, u = x[t] @ gw.T, x[t] @ uw.T
        with np.errstate(over="ignore"):
            h64 = g / (1 + np.exp(-g)) * u
        dh = np.abs(h64) * 2.0 ** -20                # expf, a division and a product in fp32
        lo, hi, h = bf16(h64 - dh), bf16(h64 + dh), bf16(h64)
        off = np.abs(hi - lo) + np.abs(h).max(1, keepdims=True) * 2.0 ** -21
        prod = np.abs(h[:, None, :] * dw[None])      # [tokens, H, I]
        blocks = prod.reshape(len(t), H, I // 16, 16).max(3).sum(2) * 2.0 ** -12
        err = blocks + prod.sum(2) * (I + 8) * 2.0 ** -24 + off @ np.abs(dw).T
        w = wts[t, j][:, None]
        ref[t] += w * (h @ dw.T)
        bound[t] += w * err
    bound += np.abs(ref) * 2.0 ** -20                # weights, combine
    assert np.all(np.abs(y - ref) <= bound), np.abs(y - ref).max(1) / bound.max(1)
    assert np.all(y[min(7, T - 1)] == 0.0)


def test_decode_block_against_the_host():
    """The same chain as above, every step against its 64-bit form on the
    previous step's device output: the projection within its fp32 sums and one
    bf16 rounding, the MLP within 2^-8 in the Frobenius norm (a bf16 rounding
    of every element is at most that, typically a third of it, which leaves
    room for the few h whose rounding the fp32 sums decide)."""
    import test_gpu_fp8 as f8
    say("block against the host")
    T, H, I = 6, 512, 640
    L = Layer(T, H, 256, 16, 4, 128, gate=True, seed=12)
    g = torch.Generator().manual_seed(5)
    ws = [native.fp8_block_quantize((torch.randn(*s, generator=g) * 0.05).to(DEV), 128)
          for s in ((H, H), (I, H), (I, H), (H, I))]
    a = native.fp8_block_linear(L.x, *ws[0])
    y, _ = L.run(x=a)
    z = native.fp8_block_mlp(y, *ws[1:])
    q, s = f8.quantize_ref(L.x.float().cpu().numpy(), 1)
    ref, mag = f8.linear_ref(q * f8.spread(s, T, H, 1), f8.values(*ws[0], 128))
    f8.check_out(a, ref, f8.sum_bound(mag, H), "projection")
    q, s = f8.quantize_ref(y.float().cpu().numpy(), 1)
    gate, up, down = (f8.values(*w, 128) for w in ws[1:])
    xv = q * f8.spread(s, T, H, 1)
    gt, ut = xv @ gate.T, xv @ up.T
    q, s = f8.quantize_ref(bf16(gt / (1 + np.exp(-gt)) * ut).astype(np.float32), 1)
    ref = (q * f8.spread(s, T, I, 1)) @ down.T
    assert np.linalg.norm(z.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
