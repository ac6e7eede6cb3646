"""FP8 block-scaled operators against plain 64-bit forms: the quantiser bit for
bit, the linear product and the gated MLP within bounds that follow from their
fp32 sums and final rounding."""
import sys

import numpy as np
import pytest
import torch

from nvfp4_routed_expert_amd import native

pytestmark = pytest.mark.gpu
DEV = "cuda"


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _blocks(n):
    return -(-n // 128)


# ---- plain forms (CPU, 64 bits; the quantiser's 32-bit steps kept) -------------


def e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    mag = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    return np.where(b & 128, -mag, mag)


def quantize_ref(x, block):
    """x fp32 numpy [R, C] -> (E4M3 values fp64, scales fp32)."""
    r, c = x.shape
    cb, rb = _blocks(c), (r if block == 1 else _blocks(r))
    pad = np.zeros((rb * block, cb * 128), np.float32)
    pad[:r, :c] = x
    pad = pad.reshape(rb, block, cb, 128)
    top = np.abs(pad).max((1, 3))
    s = np.where(top > 0, np.maximum(top / np.float32(448), np.float32(2.0 ** -126)),
                 np.float32(1)).astype(np.float32)
    inv = (np.float32(1) / s).astype(np.float32)
    v = (pad * inv[:, None, :, None]).astype(np.float32).astype(np.float64)
    a = np.minimum(np.abs(v), 448.0)
    ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -40))), -6.0) - 3.0)
    q = np.copysign(np.rint(a / ulp) * ulp, v)
    return q.reshape(rb * block, cb * 128)[:r, :c], s


def spread(s, rows, cols, block):
    s = np.repeat(s.astype(np.float64), 128, 1)[:, :cols]
    return s if block == 1 else np.repeat(s, 128, 0)[:rows]


def values(codes, s, block):
    return e4m3_table()[codes.cpu().numpy()] * spread(s.cpu().numpy(), *codes.shape, block)


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def linear_ref(xv, wv):
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def sum_bound(mag, K):
    """fp32 sums of K exact products: at most K roundings inside the blocks and
    two per block (its scale, its joining) of 2^-24 of the sum of magnitudes."""
    return mag * (K + 4 * _blocks(K)) * 2.0 ** -24


def check(y, ref, bound, what):
    y = y.double().cpu().numpy() if isinstance(y, torch.Tensor) else y
    over = np.abs(y - ref) - bound
    assert np.all(over <= 0), f"{what}: {int((over > 0).sum())} outside, worst {over.max():.3e}"


# The fp8 matrix instruction (bf16 outputs of more than 64 rows) aligns a
# block's products to the largest with about 12 bits: at most 2^-10 of the
# largest product per block is allowed for it (2^-10.9 measured over 2^17
# blocks of wide data).


def block_alignment(xv, wv):
    top = 0.0
    for b in range(0, xv.shape[1], 128):
        top = top + np.abs(xv[:, b:b + 128]).max(1)[:, None] * np.abs(wv[:, b:b + 128]).max(1)[None]
    return top * 2.0 ** -10


def check_out(y, ref, bound, what):
    """bf16 outputs: half a step of the value more (2^-8 of it, its bound included)."""
    extra = (np.abs(ref) + bound) * 2.0 ** -8 if y.dtype == torch.bfloat16 else 0.0
    check(y, ref, bound + extra, what)


def acts(rows, cols, seed, dtype=torch.bfloat16):
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(1, cols, generator=g))
    return x.to(dtype)


def weight(n, k, seed):
    w = torch.randn(n, k, generator=_gen(seed)) * 0.02
    return native.fp8_block_quantize(w.to(DEV), 128)


# ---- quantiser --------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 5120), (3, 160), (16, 128), (129, 2080),
                                       (257, 96), (300, 1056)])
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_bit_exact(rows, cols, block, dtype):
    say("quantize", rows, cols, block, dtype)
    x = acts(rows, cols, rows + cols, dtype)
    x[rows // 2, : min(cols, 128)] = 0.0                       # a zero 1 x 128 block
    codes, s = native.fp8_block_quantize(x.to(DEV), block)
    q, ref_s = quantize_ref(x.float().numpy(), block)
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(e4m3_table()[codes.cpu().numpy()], q)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_row_stride_and_extremes(block):
    """A strided view, and blocks of subnormals, of one value and of the
    largest numbers."""
    say("quantize stride", block)
    base = acts(260, 512, 5, torch.float32)
    base[0, :] = 1e-40                      # subnormal: the scale's floor
    base[1, :128] = 3e38
    base[2, :128] = torch.finfo(torch.float32).max
    base[3, 128:256] = 0.0
    base[4, 130] = -448.0 * 2.0 ** -126
    x = base.to(DEV)[:, :480]
    assert x.stride(0) == 512
    codes, s = native.fp8_block_quantize(x, block)
    q, ref_s = quantize_ref(base[:, :480].numpy(), block)
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(e4m3_table()[codes.cpu().numpy()], q)


# ---- linear -----------------------------------------------------------------------

SHAPES = [(1, 17, 32), (1, 512, 256), (2, 300, 2080), (8, 129, 128), (16, 1000, 544),
          (17, 64, 1024), (33, 255, 160), (64, 513, 512), (65, 256, 4096), (77, 500, 2080),
          (130, 640, 96), (257, 384, 1056), (1100, 300, 288)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K):
    say("linear", M, N, K)
    x = acts(M, K, M * 7 + K)
    w, ws = weight(N, K, N + K)
    xq, xs = native.fp8_block_quantize(x.to(DEV))
    q, _ = quantize_ref(x.float().numpy(), 1)
    xv, wv = q * spread(xs.cpu().numpy(), M, K, 1), values(w, ws, 128)
    ref, mag = linear_ref(xv, wv)
    bound = sum_bound(mag, K)
    y32 = native.fp8_block_linear(x.to(DEV), w, ws, out_dtype=torch.float32)
    check_out(y32, ref, bound, f"f32 {M} {N} {K}")
    y16 = native.fp8_block_linear(x.to(DEV), w, ws)
    if M <= 64:
        assert torch.equal(y16, y32.to(torch.bfloat16))
    else:
        check_out(y16, ref, bound + block_alignment(xv, wv), f"bf16 {M} {N} {K}")
    assert torch.equal(native.fp8_block_linear(xq, w, ws, x_scales=xs), y16)
    pre = native.fp8_block_linear(xq, w, ws, x_scales=xs, out_dtype=torch.float32)
    assert torch.equal(pre, y32)
    assert torch.equal(native.fp8_block_linear(x.to(DEV), w, ws, out_dtype=torch.float32), y32)


def test_linear_writes_its_rows_only():
    """Rows behind the batch and the output's neighbours keep their contents."""
    M, N, K = 5, 200, 256
    say("linear rows", M, N, K)
    w, ws = weight(N, K, 3)
    buf = torch.full((M + 4, N), 7.0, dtype=torch.float32, device=DEV)
    x = acts(M, K, 9).to(DEV)
    native.fp8_block_linear(x, w, ws, out=buf[2:2 + M])
    assert torch.all(buf[:2] == 7.0) and torch.all(buf[2 + M:] == 7.0)
    assert torch.equal(buf[2:2 + M], native.fp8_block_linear(x, w, ws, out_dtype=torch.float32))


def test_empty_batches():
    say("empty")
    w, ws = weight(64, 96, 1)
    d, ds = weight(96, 64, 2)
    x = torch.empty((0, 96), dtype=torch.bfloat16, device=DEV)
    assert native.fp8_block_linear(x, w, ws).shape == (0, 64)
    assert native.fp8_block_mlp(x, (w, ws), (w, ws), (d, ds)).shape == (0, 96)
    codes, s = native.fp8_block_quantize(x)
    assert codes.shape == (0, 96) and s.shape == (0, 1)


# ---- gated MLP ----------------------------------------------------------------------


GRID = np.array([0.0, 64.0, 128.0, 256.0, 448.0])


def grid(rows, cols, seed, exp):
    """Values on the E4M3 grid times 2^exp, each 128-block with a 448: their
    scales are exactly 2^exp, and sums of products of two such (multiples of
    2^12 below 2^18, up to 2^11 terms and more) are exact in fp32."""
    r = np.random.default_rng(seed)
    v = r.choice(GRID, (rows, cols), p=[0.3, 0.3, 0.2, 0.15, 0.05]) * r.choice([-1, 1], (rows, cols))
    v[:, ::128] = 448.0
    return (v * 2.0 ** exp).astype(np.float32)


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (1, 2048, 1056), (3, 160, 96), (16, 512, 640),
                                   (24, 2048, 1056), (40, 1024, 32), (64, 544, 2080),
                                   (70, 256, 544), (200, 640, 1024)])
def test_mlp(T, H, I):
    """Inputs whose gate and up sums are exact, so h is known up to expf: an h
    within 2^-20 of a rounding boundary may take either neighbour (and move its
    block's scale); every other h, and so every row without such an h, must
    give y to the rounding of the down sums."""
    say("mlp", T, H, I)
    x = grid(T, H, T, -8)
    raw = [grid(I, H, 1, -17), grid(I, H, 2, -17), 0.02 * np.random.default_rng(3).standard_normal(
        (H, I)).astype(np.float32)]
    mats = [native.fp8_block_quantize(torch.from_numpy(w).to(DEV), 128) for w in raw]
    assert np.array_equal(values(*mats[0], 128), raw[0].astype(np.float64))
    g, u = x.astype(np.float64) @ raw[0].T.astype(np.float64), \
        x.astype(np.float64) @ raw[1].T.astype(np.float64)
    h64 = g / (1 + np.exp(-g)) * u
    dh = np.abs(h64) * 2.0 ** -20          # expf, a division and two products in fp32
    lo, hi, h = bf16(h64 - dh), bf16(h64 + dh), bf16(h64)
    loose = lo != hi
    assert loose.mean() < 0.01
    q, s = quantize_ref(h.astype(np.float32), 1)
    down = values(*mats[2], 128)
    ref, mag = linear_ref(q * spread(s, T, I, 1), down)
    hm = np.maximum(np.abs(lo), np.abs(hi))
    pad, padl = np.zeros((T, _blocks(I) * 128)), np.zeros((T, _blocks(I) * 128), bool)
    pad[:, :I], padl[:, :I] = hm, loose
    top = np.repeat(pad.reshape(T, -1, 128).max(2), 128, 1)
    moves = (padl & (pad >= 0.98 * top)).reshape(T, -1, 128).any(2)    # may set the scale
    step = np.where(np.repeat(moves, 128, 1)[:, :I] | loose,
                    hm * 2.0 ** -3 + top[:, :I] * 2.0 ** -17, 0.0)     # one E4M3 step
    bound = sum_bound(mag, I) * 1.01 + step @ np.abs(down).T
    xd = torch.from_numpy(x).to(torch.bfloat16).to(DEV)
    y32 = native.fp8_block_mlp(xd, *mats, out_dtype=torch.float32)
    check_out(y32, ref, bound, f"mlp {T} {H} {I}")
    y16 = native.fp8_block_mlp(xd, *mats)
    if T <= 64:
        assert torch.equal(y16, y32.to(torch.bfloat16))
    else:
        check_out(y16, ref, bound + block_alignment(q * spread(s, T, I, 1), down), "bf16 mlp")
    assert torch.equal(native.fp8_block_mlp(xd, *mats, out_dtype=torch.float32), y32)


def test_mlp_random_inputs():
    """Gaussian inputs: bf16 outputs within 2^-8 of the 64-bit form in the
    Frobenius norm (half a bf16 step of every element at most 2^-8 relative;
    typically a third of it, which leaves room for the few h whose rounding
    the fp32 sums decide)."""
    T, H, I = 24, 1024, 1056
    say("mlp random", T, H, I)
    x = acts(T, H, 5)
    mats = [weight(I, H, 11), weight(I, H, 12), weight(H, I, 13)]
    q, s = quantize_ref(x.float().numpy(), 1)
    gate, up, down = (values(*m, 128) for m in mats)
    xv = q * spread(s, T, H, 1)
    g, u = xv @ gate.T, xv @ up.T
    q, s = quantize_ref(bf16(g / (1 + np.exp(-g)) * u).astype(np.float32), 1)
    ref = (q * spread(s, T, I, 1)) @ down.T
    y = native.fp8_block_mlp(x.to(DEV), *mats).double().cpu().numpy()
    assert np.linalg.norm(y - ref) <= 2.0 ** -8 * np.linalg.norm(ref)


# ---- graphs, streams ----------------------------------------------------------------


@pytest.mark.parametrize("T", [4, 100])
def test_linear_and_mlp_in_a_graph(T):
    """Captured and replayed with eager work between the replays: every replay
    equals the eager result on the same inputs."""
    H, I = 512, 640
    say("graph", T)
    mats = [weight(I, H, 21), weight(I, H, 22), weight(H, I, 23)]
    x = acts(T, H, 31).to(DEV)
    y, z = torch.empty_like(x), torch.empty((T, I), dtype=torch.float32, device=DEV)
    L = native.lib()
    wl = torch.empty(L.fp8_block_linear_workspace_size(T, I, H, 0), dtype=torch.uint8, device=DEV)
    wm = torch.empty(L.fp8_block_mlp_workspace_size(T, H, I), dtype=torch.uint8, device=DEV)

    def step():
        native.fp8_block_mlp(x, *mats, out=y, workspace=wm)
        native.fp8_block_linear(y, *mats[0], out=z, workspace=wl)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(4):
        x.copy_(acts(T, H, 40 + seed))
        want_y = native.fp8_block_mlp(x, *mats)
        want_z = native.fp8_block_linear(want_y, *mats[0], out_dtype=torch.float32)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(z, want_z)


# ---- where the forms change ---------------------------------------------------------


@pytest.mark.parametrize("M,N,K", [(1, 33, 18432), (4, 70, 4864), (4, 70, 5120), (9, 30, 18432),
                                   (24, 4096, 1024), (24, 4112, 1024), (32, 48, 1536),
                                   (32, 48, 1568), (64, 31, 18432), (65, 257, 160),
                                   (129, 1003, 640), (193, 515, 4224), (385, 130, 512)])
def test_linear_at_the_rules(M, N, K):
    """Either side of the rules: x quantised inside (small, large, a workgroup
    per CU) or by a launch, few rows or a batch, odd columns, K parts that are
    not whole groups of blocks."""
    test_linear(M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 40, 18464), (33, 130, 18560), (17, 8192, 5888),
                                   (33, 8192, 3936)])
def test_linear_of_few_rows_with_a_long_k(M, N, K):
    """Past the few-row form's K, and with large weights, the batch form runs,
    exact for either type."""
    test_linear(M, N, K)


@pytest.mark.parametrize("T,H,I", [(2, 64, 18464), (2, 18464, 32), (8, 1024, 1056), (17, 2048, 96),
                                   (32, 1568, 160)])
def test_mlp_at_the_rules(T, H, I):
    test_mlp(T, H, I)


def test_row_of_infinite_scale_stays_alone():
    """A token with non-finite values: its own row is not finite, the others
    are as without it."""
    say("linear infinite row")
    for M in (3, 20, 100):
        w, ws = weight(96, 640, 5)
        x = acts(M, 640, M).to(DEV)
        clean = native.fp8_block_linear(x, w, ws, out_dtype=torch.float32)
        x[1, 7] = float("inf")
        y = native.fp8_block_linear(x, w, ws, out_dtype=torch.float32)
        keep = torch.ones(M, dtype=torch.bool, device=DEV)
        keep[1] = False
        assert torch.equal(y[keep], clean[keep])
        assert not torch.isfinite(y[1]).any()


def test_linear_on_two_streams_at_once():
    say("linear two streams")
    w, ws = weight(1000, 2080, 8)
    xs_ = [acts(77, 2080, s).to(DEV) for s in (1, 2)]
    want = [native.fp8_block_linear(x, w, ws, out_dtype=torch.float32) for x in xs_]
    streams = [torch.cuda.Stream() for _ in xs_]
    got = []
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x in zip(streams, xs_):
            with torch.cuda.stream(s):
                got.append(native.fp8_block_linear(x, w, ws, out_dtype=torch.float32))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("M", [1, 6])
def test_large_weights_equal_their_parts(M):
    """Weights past the size from which they are loaded as used once: rows of W,
    and columns of h, as with the parts alone (bit for bit)."""
    H, I, part = 5120, 13056, 384
    say("large weights", M)
    gen = torch.Generator(device=DEV).manual_seed(M)
    quant = lambda r, c: native.fp8_block_quantize(
        0.02 * torch.randn(r, c, generator=gen, device=DEV), 128)
    x = acts(M, H, 3).to(DEV)
    w, ws = quant(2 * I, H)
    y = native.fp8_block_linear(x, w, ws)
    assert torch.equal(y[:, -part:], native.fp8_block_linear(x, w[-part:].contiguous(),
                                                             ws[-part // 128:].contiguous()))
    gate, up = (w[:I], ws[:I // 128]), (w[I:], ws[I // 128:])
    d, ds = quant(H, I)
    d[:, part:] = 0
    whole = native.fp8_block_mlp(x, gate, up, (d, ds))
    cut = lambda m: (m[0][:part].contiguous(), m[1][:part // 128].contiguous())
    alone = native.fp8_block_mlp(x, cut(gate), cut(up), (d[:, :part].contiguous(),
                                                         ds[:, :part // 128].contiguous()))
    assert torch.equal(whole, alone)


@pytest.mark.parametrize("N,K,rows", [(640, 4096, (455, 384, 385, 130, 65, 64, 20, 1)),
                                      (130, 18560, (150, 64, 65, 33, 2))])
@pytest.mark.parametrize("pre", [False, True])
def test_workspace_of_the_largest_batch(N, K, rows, pre):
    """One workspace, of the first batch's size, for the smaller ones (whose K
    is split further, or whose form is another): the results of a call that
    makes its own."""
    say("workspace linear", N, K, pre)
    w, ws = weight(N, K, 41)
    size = native.lib().fp8_block_linear_workspace_size
    space = torch.empty(size(rows[0], N, K, pre), dtype=torch.uint8, device=DEV)
    x = acts(rows[0], K, 42).to(DEV)
    q, s = native.fp8_block_quantize(x)
    for M in rows:
        for dt in (torch.float32, torch.bfloat16):
            a = (q[:M], w, ws, s[:M].contiguous()) if pre else (x[:M], w, ws)
            got = native.fp8_block_linear(*a, out_dtype=dt, workspace=space)
            assert torch.equal(got, native.fp8_block_linear(*a, out_dtype=dt))


@pytest.mark.parametrize("H,I,rows", [(512, 2080, (260, 200, 70, 65, 64, 33, 32, 1)),
                                      (2080, 544, (130, 66, 40, 17, 5))])
def test_mlp_workspace_of_the_largest_batch(H, I, rows):
    say("workspace mlp", H, I)
    mats = [weight(I, H, 51), weight(I, H, 52), weight(H, I, 53)]
    space = torch.empty(native.lib().fp8_block_mlp_workspace_size(rows[0], H, I),
                        dtype=torch.uint8, device=DEV)
    x = acts(rows[0], H, 54).to(DEV)
    for T in rows:
        for dt in (torch.float32, torch.bfloat16):
            got = native.fp8_block_mlp(x[:T], *mats, out_dtype=dt, workspace=space)
            assert torch.equal(got, native.fp8_block_mlp(x[:T], *mats, out_dtype=dt))


# ---- the larger tiles ---------------------------------------------------------------

# bf16 products whose tiles have 128 and 192 rows, with K whole and in parts:
# (M, N, K, rows of a tile, parts).  Last tiles of one row and of all but one,
# odd N, K with a last block of 32, 96 and 128 columns, odd and even numbers of
# blocks, parts of different lengths.
TILE_SHAPES = [(257, 13777, 160, 128, 1), (383, 10787, 416, 128, 1), (257, 13777, 1056, 128, 1),
               (300, 17408, 128, 128, 1), (385, 16399, 160, 192, 1), (575, 13349, 416, 192, 1),
               (577, 13351, 288, 192, 1), (385, 17301, 736, 192, 1), (512, 17408, 512, 192, 1),
               (2057, 34, 3968, 128, 8), (1602, 34, 4640, 128, 10), (645, 3841, 12192, 192, 4),
               (2719, 33, 6048, 192, 12)]
# (T, H, I, rows of a tile, parts) of the gate and up products
MLP_TILE_SHAPES = [(65, 160, 16416, 128, 1), (191, 1056, 11008, 128, 1), (129, 32, 16416, 192, 1),
                   (385, 160, 8224, 192, 1), (191, 96, 16416, 192, 1), (67, 4640, 5504, 128, 5),
                   (65, 5312, 5664, 128, 4), (1345, 12160, 928, 192, 4)]


@pytest.mark.parametrize("M,N,K,rows,parts", TILE_SHAPES)
def test_linear_of_larger_tiles(M, N, K, rows, parts):
    assert native.fp8_debug_plan(M, N, K) == (rows, parts)
    test_linear(M, N, K)


@pytest.mark.parametrize("T,H,I,rows,parts", MLP_TILE_SHAPES)
def test_mlp_of_larger_tiles(T, H, I, rows, parts):
    assert native.fp8_debug_plan(T, I, H, gate_up=True) == (rows, parts)
    test_mlp(T, H, I)


def test_rows_behind_a_larger_tile_are_left():
    """A last tile of one row stores that row alone, bf16 and f32 parts."""
    for M, N, K, rows, parts in ((257, 13777, 160, 128, 1), (385, 16399, 160, 192, 1),
                                 (1345, 34, 4640, 64, 10)):
        say("rows behind", M, N, K)
        assert native.fp8_debug_plan(M, N, K) == (rows, parts)
        w, ws = weight(N, K, 61)
        x = acts(M, K, 62).to(DEV)
        base = torch.full((M + 64, N), 7.0, dtype=torch.bfloat16, device=DEV)
        out = base[:M]
        native.fp8_block_linear(x, w, ws, out=out)
        assert torch.all(base[M:] == 7.0)
        assert torch.equal(out, native.fp8_block_linear(x, w, ws))
