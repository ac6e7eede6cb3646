"""int8 quantiser, linear product and gated MLP against plain 64-bit forms.  The
sums are integers and every later step is one fp32 operation, so the quantiser
and the product are compared bit for bit."""
import sys
import threading

import numpy as np
import pytest
import torch

from nvfp4_routed_expert_amd import native

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = np.float32


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- plain forms (CPU; the 32-bit steps of the definitions kept) ---------------


def quantize_ref(x):
    """x fp32 numpy [R, C] -> (int64 codes, fp32 scales)."""
    top = np.abs(x).max(1)
    s = np.where(top > 0, np.maximum(top / F32(127), F32(2.0 ** -126)), F32(1)).astype(F32)
    inv = (F32(1) / s).astype(F32)
    return np.rint((x * inv[:, None]).astype(F32)).astype(np.int64), s


def linear_ref(xq, xs, wq, ws):
    """fp32 [M, N]; sums in 64 bits (integers below 2^53: exact)."""
    acc = (xq.astype(np.float64) @ wq.T.astype(np.float64)).astype(F32)
    return ((acc * xs[:, None]).astype(F32) * ws[None, :]).astype(F32)


def bf16(x):
    return torch.from_numpy(np.asarray(x, F32)).to(torch.bfloat16)


def acts(rows, cols, seed, dtype=torch.bfloat16):
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(1, cols, generator=g))
    return x.to(dtype)


def codes(n, k, seed):
    """Any codes (-128 among them) and positive scales."""
    g = _gen(seed)
    q = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    return q, torch.rand(n, generator=g) * 1e-3 + 1e-4


def same(y, ref, what):
    """Bit for bit (bf16: the rounded fp32 result)."""
    want = torch.from_numpy(ref)
    if y.dtype == torch.bfloat16:
        want = want.to(torch.bfloat16)
    bad = (y.cpu() != want).sum().item()
    assert bad == 0, f"{what}: {bad} of {want.numel()} differ"


# ---- quantiser --------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 5120), (3, 160), (16, 128), (129, 2080),
                                       (257, 96), (300, 1056), (5, 512), (5, 544), (3, 1024),
                                       (3, 1056), (2, 8192), (2, 8224), (2, 17408), (2, 32768),
                                       (2, 32800), (3, 131040), (1000, 32)])
def test_quantize_bit_exact(rows, cols, dtype):
    say("quantize", rows, cols, dtype)
    x = acts(rows, cols, rows + cols, dtype)
    x[rows // 2] = 0.0                                          # a zero row
    if rows > 2:
        x[0, -1] = 300.0                                        # the maximum in a last column
        x[-1, 0] = -500.0
    q, s = native.int8_quantize(x.to(DEV))
    ref, ref_s = quantize_ref(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(q.cpu().numpy(), ref)


def test_quantize_row_stride_ties_and_extremes():
    say("quantize stride")
    base = acts(40, 512, 5, torch.float32)
    base[0, :] = 1e-40                      # subnormal: the scale's floor
    base[1, :128] = 3e38
    base[2, :128] = torch.finfo(torch.float32).max
    base[3, :] = 0.0
    base[4, 130] = -448.0 * 2.0 ** -126
    base[5, :] = torch.arange(512) % 127 + 0.5       # ties
    base[5, 7] = 127.0
    base[6, :] = -0.0
    base[6, 3] = 127.0
    x = base.to(DEV)[:, :480]
    assert x.stride(0) == 512
    q, s = native.int8_quantize(x)
    ref, ref_s = quantize_ref(base[:, :480].numpy())
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(q.cpu().numpy(), ref)
    y = base.to(torch.bfloat16).to(DEV)[3:, 16:112]
    q, s = native.int8_quantize(y)
    ref, ref_s = quantize_ref(y.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ref_s) and np.array_equal(q.cpu().numpy(), ref)


# ---- linear -----------------------------------------------------------------------

SHAPES = [(1, 17, 32), (1, 512, 256), (2, 300, 2080), (8, 129, 128), (16, 1000, 544),
          (17, 64, 1024), (33, 255, 160), (64, 513, 512), (65, 256, 4096), (77, 500, 2080),
          (130, 640, 96), (257, 384, 1056), (1100, 300, 288), (3, 1, 64), (200, 1, 32),
          (5, 4100, 8224), (70, 33, 17408), (129, 130, 224)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K):
    say("linear", M, N, K)
    x = acts(M, K, M * 7 + K)
    w, ws = codes(N, K, N + K)
    q, s = quantize_ref(x.float().numpy())
    ref = linear_ref(q, s, w.numpy(), ws.numpy())
    w, ws, xd = w.to(DEV), ws.to(DEV), x.to(DEV)
    y32 = native.int8_linear(xd, w, ws, out_dtype=torch.float32)
    same(y32, ref, f"f32 {M} {N} {K}")
    same(native.int8_linear(xd, w, ws), ref, f"bf16 {M} {N} {K}")
    xq, xs = native.int8_quantize(xd)
    same(native.int8_linear(xq, w, ws, x_scales=xs), ref, f"codes bf16 {M} {N} {K}")
    same(native.int8_linear(xq, w, ws, x_scales=xs, out_dtype=torch.float32), ref,
         f"codes f32 {M} {N} {K}")


@pytest.mark.parametrize("M", [1, 20, 150])
def test_linear_largest_sums(M):
    """All codes -128 over the longest K: the sum is 2^31 - 2^19, of either sign."""
    K, N = 131040, 40
    say("linear largest", M)
    x = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    one = torch.ones(max(M, N), device=DEV)
    y = native.int8_linear(x, w, one[:N], x_scales=one[:M], out_dtype=torch.float32)
    assert (y[:, ::2] == float(K * 128 * 128)).all()
    assert (y[:, 1::2] == float(F32(-K * 128 * 127))).all()


def test_linear_small_and_large_scales():
    """The sum meets s_x before s_w: scales whose product alone would vanish."""
    say("linear scales")
    x, w = codes(3, 64, 1)[0], codes(50, 64, 2)[0]
    for sx, sw in ((1e-25, 1e-18), (1e-18, 1e-25), (1e30, 1e-30), (2e20, 1e15), (0.0, 1.0)):
        xs, ws = np.full(3, sx, F32), np.full(50, sw, F32)
        y = native.int8_linear(x.to(DEV), w.to(DEV), torch.from_numpy(ws).to(DEV),
                               x_scales=torch.from_numpy(xs).to(DEV), out_dtype=torch.float32)
        same(y, linear_ref(x.numpy(), xs, w.numpy(), ws), f"{sx} {sw}")


@pytest.mark.parametrize("M,N,K", [(5, 200, 256), (70, 300, 160), (300, 257, 288)])
def test_linear_writes_its_rows_only(M, N, K):
    """Rows before and behind the batch keep their contents."""
    say("linear rows", M, N, K)
    w, ws = (t.to(DEV) for t in codes(N, K, 3))
    x = acts(M, K, 9).to(DEV)
    for dt in (torch.float32, torch.bfloat16):
        want = native.int8_linear(x, w, ws, out_dtype=dt)
        buf = torch.full((M + 16, N), 7.0, dtype=dt, device=DEV)
        native.int8_linear(x, w, ws, out=buf[8:8 + M])
        assert torch.all(buf[:8] == 7.0) and torch.all(buf[8 + M:] == 7.0)
        assert torch.equal(buf[8:8 + M], want)


def test_empty_batches():
    say("empty")
    w, ws = (t.to(DEV) for t in codes(64, 96, 1))
    d, ds = (t.to(DEV) for t in codes(96, 64, 2))
    x = torch.empty((0, 96), dtype=torch.bfloat16, device=DEV)
    assert native.int8_linear(x, w, ws).shape == (0, 64)
    assert native.int8_mlp(x, (w, ws), (w, ws), (d, ds)).shape == (0, 96)
    q, s = native.int8_quantize(x)
    assert q.shape == (0, 96) and s.shape == (0,)


def test_row_of_infinite_scale_stays_alone():
    """A token with a non-finite value: the others are as without it."""
    say("linear infinite row")
    for M in (3, 20, 100):
        w, ws = (t.to(DEV) for t in codes(96, 640, 5))
        x = acts(M, 640, M).to(DEV)
        clean = native.int8_linear(x, w, ws, out_dtype=torch.float32)
        x[1, 7] = float("inf")
        y = native.int8_linear(x, w, ws, out_dtype=torch.float32)
        keep = torch.ones(M, dtype=torch.bool, device=DEV)
        keep[1] = False
        assert torch.equal(y[keep], clean[keep])


# ---- gated MLP ----------------------------------------------------------------------


def mlp_ref(xq, xs, gate, up, down):
    """(ref, bound) of y in 64 bits.  gate and up are known to the bit, h up to
    expf, a division and two products: an h within 2^-20 of a rounding boundary
    may take either neighbour.  One bf16 step is at most 127 / 128 of a code, so
    it moves a code by at most one; where it may be the row's maximum, the scale
    moves by up to 2^-7 of itself and every code by at most one.  Rows without
    such an h have bound 0: they are exact."""
    g = linear_ref(xq, xs, *gate).astype(np.float64)
    u = linear_ref(xq, xs, *up).astype(np.float64)
    h64 = g / (1 + np.exp(-g)) * u
    dh = np.abs(h64) * 2.0 ** -20
    lo, hi = bf16(h64 - dh).float().numpy(), bf16(h64 + dh).float().numpy()
    h = bf16(h64).float().numpy()
    loose = lo != hi
    q, s = quantize_ref(h)
    ref = linear_ref(q, s, *down)
    top = np.abs(h).max(1, keepdims=True)
    moves = (loose & (np.abs(h) >= 0.98 * top)).any(1, keepdims=True)
    per = np.where(moves, 1.01 + np.abs(q) * 2.0 ** -7, np.where(loose, 1.0, 0.0)) * s[:, None]
    wd = np.abs(down[0].astype(np.float64)) * down[1][:, None]
    mag = np.abs(ref)
    bound = per @ wd.T
    return ref, np.where(loose.any(1, keepdims=True), bound + 2.0 ** -21 * (mag + bound), 0.0), loose


MLP_SHAPES = [(1, 256, 128), (1, 2048, 1056), (3, 160, 96), (16, 512, 640), (24, 2048, 1056),
              (40, 1024, 32), (64, 544, 2080), (70, 256, 544), (200, 640, 1024), (300, 96, 288),
              (2, 5120, 8224)]


@pytest.mark.parametrize("T,H,I", MLP_SHAPES)
def test_mlp(T, H, I):
    say("mlp", T, H, I)
    x = acts(T, H, T)
    mats = [codes(*shape, seed) for seed, shape in ((1, (I, H)), (2, (I, H)), (3, (H, I)))]
    # (scales that bring gate and up to about 1)
    for w, s in mats:
        s *= 1.0 / (0.05 * w.shape[1] ** 0.5)
    host = [(w.numpy(), s.numpy()) for w, s in mats]
    dev = [(w.to(DEV), s.to(DEV)) for w, s in mats]
    xq, xs = quantize_ref(x.float().numpy())
    ref, bound, loose = mlp_ref(xq, xs, *host)
    assert loose.mean() < 0.01
    xd = x.to(DEV)
    y = native.int8_mlp(xd, *dev, out_dtype=torch.float32)
    over = np.abs(y.double().cpu().numpy() - ref) - bound
    assert (over <= 0).all(), f"{(over > 0).sum()} outside, worst {over.max()}"
    assert torch.equal(native.int8_mlp(xd, *dev), y.to(torch.bfloat16))
    q, s = native.int8_quantize(xd)
    assert torch.equal(native.int8_mlp(q, *dev, x_scales=s, out_dtype=torch.float32), y)


# ---- graphs, streams, workspaces -------------------------------------------------------


@pytest.mark.parametrize("T", [4, 100])
def test_linear_and_mlp_in_a_graph(T):
    """Captured and replayed with eager work between the replays: every replay
    equals the eager result on the same inputs."""
    H, I = 512, 640
    say("graph", T)
    mats = [tuple(t.to(DEV) for t in codes(*sh, seed))
            for seed, sh in ((21, (I, H)), (22, (I, H)), (23, (H, I)))]
    x = acts(T, H, 31).to(DEV)
    y, z = torch.empty_like(x), torch.empty((T, I), dtype=torch.float32, device=DEV)
    L = native.lib()
    space = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)
    wl = space(L.int8_linear_workspace_size(T, I, H, 0))
    wm = space(L.int8_mlp_workspace_size(T, H, I, 0))

    def step():
        native.int8_mlp(x, *mats, out=y, workspace=wm)
        native.int8_linear(y, *mats[0], out=z, workspace=wl)

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
        want_y = native.int8_mlp(x, *mats)
        want_z = native.int8_linear(want_y, *mats[0], out_dtype=torch.float32)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(z, want_z)


def test_linear_on_two_streams_at_once():
    say("linear two streams")
    for M in (6, 77, 300):
        w, ws = (t.to(DEV) for t in codes(1000, 2080, 8))
        xs_ = [acts(M, 2080, s).to(DEV) for s in (1, 2)]
        want = [native.int8_linear(x, w, ws, out_dtype=torch.float32) for x in xs_]
        streams = [torch.cuda.Stream() for _ in xs_]
        got = []
        torch.cuda.synchronize()
        for _ in range(5):
            for s, x in zip(streams, xs_):
                with torch.cuda.stream(s):
                    got.append(native.int8_linear(x, w, ws, out_dtype=torch.float32))
        torch.cuda.synchronize()
        for i, y in enumerate(got):
            assert torch.equal(y, want[i % 2])


def test_two_graphs_share_a_workspace():
    """Two captured products in parts of K on one workspace, replayed in turn."""
    say("graphs on one workspace")
    N, K = 1000, 4128
    sizes = (40, 130)
    assert all(native.int8_debug_plan(M, N, K)[2] > 1 for M in sizes)
    w, ws = (t.to(DEV) for t in codes(N, K, 71))
    space = torch.full((native.lib().int8_linear_workspace_size(max(sizes), N, K, 0),), 0xFF,
                       dtype=torch.uint8, device=DEV)
    x = [acts(M, K, M).to(DEV) for M in sizes]
    y = [torch.empty((M, N), dtype=torch.float32, device=DEV) for M in sizes]
    graphs = []
    for i in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            native.int8_linear(x[i], w, ws, out=y[i], workspace=space)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            native.int8_linear(x[i], w, ws, out=y[i], workspace=space)
        graphs.append(g)
    for seed in range(3):
        for i, M in enumerate(sizes):
            x[i].copy_(acts(M, K, 80 + seed + 10 * i))
        want = [native.int8_linear(v, w, ws, out_dtype=torch.float32) for v in x]
        torch.cuda.synchronize()
        for i in (0, 1, 0):
            y[i].fill_(7.0)
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y, want))


def test_calls_from_two_threads():
    """Each thread on a stream of its own; also its refusals are its own."""
    say("two threads")
    H, I = 1024, 672
    mats = [tuple(t.to(DEV) for t in codes(*sh, seed))
            for seed, sh in ((61, (I, H)), (62, (I, H)), (63, (H, I)))]
    xs = [acts(T, H, T).to(DEV) for T in (3, 90)]
    want = [native.int8_mlp(x, *mats) for x in xs]
    torch.cuda.synchronize()
    got, errors = [[], []], [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(8):
                got[i].append(native.int8_mlp(xs[i], *mats))
                try:
                    native.int8_linear(xs[i], *mats[0], out=xs[i][:, :I].contiguous().view(-1, I),
                                       workspace=torch.empty(16, dtype=torch.uint8, device=DEV)
                                       if i else None)
                except Exception as e:
                    errors[i].append(str(e))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    assert errors[0] == [] and len(errors[1]) == 8 and all("workspace" in e for e in errors[1])


@pytest.mark.parametrize("N,K,rows", [(640, 4096, (455, 384, 385, 130, 65, 64, 20, 1)),
                                      (130, 18560, (150, 64, 65, 33, 2))])
@pytest.mark.parametrize("pre", [False, True])
def test_workspace_of_the_largest_batch(N, K, rows, pre):
    """One workspace, of the first batch's size, for the smaller ones, whatever
    it held before: the results of a call that makes its own."""
    say("workspace linear", N, K, pre)
    w, ws = (t.to(DEV) for t in codes(N, K, 41))
    size = native.lib().int8_linear_workspace_size
    space = torch.full((size(rows[0], N, K, pre),), 0xFF, dtype=torch.uint8, device=DEV)
    x = acts(rows[0], K, 42).to(DEV)
    q, s = native.int8_quantize(x)
    for M in rows:
        for dt in (torch.float32, torch.bfloat16):
            a = (q[:M], w, ws, s[:M].contiguous()) if pre else (x[:M], w, ws)
            got = native.int8_linear(*a, out_dtype=dt, workspace=space)
            assert torch.equal(got, native.int8_linear(*a, out_dtype=dt))


@pytest.mark.parametrize("H,I,rows", [(512, 2080, (260, 200, 70, 65, 64, 33, 32, 1)),
                                      (2080, 544, (130, 66, 40, 17, 5)),
                                      (4128, 672, (260, 100, 65, 40, 33)),
                                      (640, 4128, (260, 100, 65, 40, 33))])
def test_mlp_workspace_of_the_largest_batch(H, I, rows):
    say("workspace mlp", H, I)
    mats = [tuple(t.to(DEV) for t in codes(*sh, seed))
            for seed, sh in ((51, (I, H)), (52, (I, H)), (53, (H, I)))]
    space = torch.full((native.lib().int8_mlp_workspace_size(rows[0], H, I, 0),), 0xFF,
                       dtype=torch.uint8, device=DEV)
    x = acts(rows[0], H, 54).to(DEV)
    for T in rows:
        for dt in (torch.float32, torch.bfloat16):
            got = native.int8_mlp(x[:T], *mats, out_dtype=dt, workspace=space)
            assert torch.equal(got, native.int8_mlp(x[:T], *mats, out_dtype=dt))


# ---- a run of them together -------------------------------------------------------------


@pytest.mark.parametrize("T", [1, 7, 90])
def test_a_dense_block(T):
    """Residual stream -> norm -> int8 projection -> norm -> int8 MLP -> stream,
    and an FP8 projection of the same norm: each call on the codes of the one
    before equals the call on the formula's."""
    H, I, N = 640, 1056, 384
    say("block", T)
    scaled = lambda n, k, seed: (lambda w, s: (w, s / (0.05 * k ** 0.5)))(*codes(n, k, seed))
    proj, gate, up, down = (scaled(*sh, 60 + i) for i, sh in
                            enumerate(((H, H), (I, H), (I, H), (H, I))))
    on = lambda m: tuple(t.to(DEV) for t in m)
    host = lambda m: tuple(t.numpy() for t in m)
    stream, x = acts(T, H, 1, torch.float32), acts(T, H, 2)
    w1, w2 = acts(1, H, 3)[0], acts(1, H, 4, torch.float32)[0]

    def norm_ref(v, w):
        r = (1.0 / np.sqrt((v.astype(np.float64) ** 2).mean(1) + 1e-6)).astype(F32)
        return ((v * r[:, None]).astype(F32) * w[None, :]).astype(F32)

    a = native.rms_norm_quantize(x.to(DEV), w1.to(DEV), residual=stream.to(DEV), codes="int8")
    v = (x.float() + stream).numpy()
    q, s = quantize_ref(norm_ref(v, w1.float().numpy()))
    assert np.array_equal(a.residual.cpu().numpy(), v)
    assert np.array_equal(a.codes.cpu().numpy(), q) and np.array_equal(a.scales.cpu().numpy(), s)
    p = native.int8_linear(a.codes, *on(proj), x_scales=a.scales)
    p_ref = linear_ref(q, s, *host(proj))
    same(p, p_ref, "projection")
    b = native.rms_norm_quantize(p, w2.to(DEV), residual=a.residual, codes="int8",
                                 y_dtype=torch.bfloat16,
                                 out=native.RmsNorm(None, None, None, a.residual))
    v = v + bf16(p_ref).float().numpy()
    n = norm_ref(v, w2.numpy())
    q, s = quantize_ref(n)
    assert b.residual is a.residual and np.array_equal(b.residual.cpu().numpy(), v)
    assert np.array_equal(b.codes.cpu().numpy(), q)
    assert torch.equal(b.y.cpu(), bf16(n))
    y = native.int8_mlp(b.codes, on(gate), on(up), on(down), x_scales=b.scales,
                        out_dtype=torch.float32)
    ref, bound, _ = mlp_ref(q, s, host(gate), host(up), host(down))
    assert (np.abs(y.double().cpu().numpy() - ref) <= bound).all()
    f = native.rms_norm_quantize(b.residual, w2.to(DEV), codes="fp8")
    w8 = native.fp8_block_quantize(torch.from_numpy(host(proj)[0][:N].astype(F32)).to(DEV), 128)
    got = native.fp8_block_linear(f.codes, *w8, x_scales=f.scales)
    again = native.fp8_block_quantize(torch.from_numpy(n).to(DEV))
    assert torch.equal(f.codes, again[0]) and torch.equal(f.scales, again[1])
    assert torch.equal(got, native.fp8_block_linear(again[0], *w8, x_scales=again[1]))


# ---- every tile of the batch form ------------------------------------------------------

# (M, N, K, rows of x of a tile, rows of W, parts): every tile with K whole and
# in parts, last tiles of one row and of all but one, odd N, K with a last block
# of 32, 64, 96 and 128 columns, parts of different lengths.
TILE_SHAPES = [(129, 19, 32, 64, 64, 1), (63, 23, 64, 64, 64, 1), (193, 25, 3232, 64, 64, 13),
               (63, 31, 3264, 64, 64, 13), (513, 1797, 32, 64, 128, 1),
               (511, 2389, 64, 64, 128, 1), (513, 585, 8288, 64, 128, 5),
               (511, 689, 10688, 64, 128, 5), (513, 6581, 32, 64, 256, 1),
               (319, 10881, 64, 64, 256, 1), (63, 16845, 9600, 64, 256, 3),
               (257, 4295, 9184, 64, 256, 3), (1025, 1929, 32, 128, 128, 1),
               (639, 3449, 64, 128, 128, 1), (641, 521, 12192, 128, 128, 8),
               (127, 8751, 8000, 128, 128, 3), (383, 19401, 448, 128, 256, 1),
               (513, 11823, 1120, 128, 256, 1), (255, 10289, 8064, 128, 256, 3),
               (257, 4313, 10208, 128, 256, 5), (767, 2911, 2144, 192, 64, 1),
               (577, 3311, 1344, 192, 64, 1), (191, 3829, 11680, 192, 64, 4),
               (961, 1319, 10016, 192, 64, 2), (769, 5295, 1248, 192, 128, 1),
               (767, 7327, 992, 192, 128, 1), (959, 1465, 9632, 192, 128, 4),
               (961, 1459, 10976, 192, 128, 3), (961, 9253, 160, 192, 256, 1),
               (575, 17179, 7840, 192, 256, 1), (191, 12481, 11712, 192, 256, 5),
               (769, 3933, 11648, 192, 256, 3), (2049, 6073, 672, 256, 256, 1),
               (1279, 9783, 704, 256, 256, 1), (255, 16761, 11648, 256, 256, 3),
               (1025, 5985, 12480, 256, 256, 2)]
# (T, I, H, ...) of the gate and up products
MLP_TILE_SHAPES = [(65, 32, 32, 64, 128, 1), (63, 32, 64, 64, 128, 1),
                   (65, 32, 1568, 64, 128, 13), (63, 32, 1600, 64, 128, 13),
                   (129, 8288, 32, 64, 256, 1), (319, 5568, 64, 64, 256, 1),
                   (63, 8352, 9600, 64, 256, 3), (1025, 992, 32, 128, 128, 1),
                   (1023, 1056, 64, 128, 128, 1), (129, 1824, 4000, 128, 128, 4),
                   (127, 7392, 12928, 128, 128, 2), (511, 7296, 512, 128, 256, 1),
                   (641, 4640, 1280, 128, 256, 1), (66, 8768, 10304, 128, 256, 3),
                   (127, 8768, 12384, 128, 256, 3), (383, 5696, 320, 192, 128, 1),
                   (961, 2208, 736, 192, 128, 1), (383, 2560, 10272, 192, 128, 3),
                   (385, 1696, 9088, 192, 128, 3), (577, 7776, 1184, 192, 256, 1),
                   (767, 6464, 1120, 192, 256, 1), (769, 2784, 12384, 192, 256, 2),
                   (1279, 5120, 704, 256, 256, 1), (1281, 5088, 800, 256, 256, 1),
                   (255, 8352, 11264, 256, 256, 3), (769, 2464, 12992, 256, 256, 3)]


def dev_codes(n, k, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8, device=DEV)
    return q, (torch.rand(n, generator=g, device=DEV) * 1e-3 + 1e-4) * scale


def dev_linear(x, xs, w, ws):
    """As linear_ref, on the device (64-bit sums of integers: exact)."""
    return ((x.double() @ w.double().t()).float() * xs[:, None]) * ws[None, :]


@pytest.mark.parametrize("M,N,K,rows,columns,parts", TILE_SHAPES)
def test_linear_of_every_tile(M, N, K, rows, columns, parts):
    say("tile", M, N, K)
    assert native.int8_debug_plan(M, N, K) == (rows, columns, parts, N)
    (x, xs), (w, ws) = dev_codes(M, K, M), dev_codes(N, K, N)
    ref = dev_linear(x, xs, w, ws)
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full(((M + rows) * N,), 7.0, dtype=dt, device=DEV)   # (rows behind the last)
        out = buf[:M * N].view(M, N)
        native.int8_linear(x, w, ws, x_scales=xs, out=out)
        assert torch.equal(out, ref.to(dt)) and torch.all(buf[M * N:] == 7.0)


@pytest.mark.parametrize("T,I,H,rows,columns,parts", MLP_TILE_SHAPES)
def test_mlp_of_every_tile(T, I, H, rows, columns, parts):
    """As test_mlp, on the device: an h whose rounding expf may decide moves its
    code by at most one (or, as the row's maximum, all by one and the scale by
    2^-7)."""
    say("mlp tile", T, I, H)
    assert native.int8_debug_plan(T, I, H, gate_up=True) == (rows, columns, parts, I)
    x, xs = dev_codes(T, H, T)
    gate, up, down = (dev_codes(n, k, s, 20.0 / k ** 0.5)
                      for s, (n, k) in ((1, (I, H)), (2, (I, H)), (3, (H, I))))
    xs = xs * 100
    g, u = dev_linear(x, xs, *gate).double(), dev_linear(x, xs, *up).double()
    h64 = g / (1 + torch.exp(-g)) * u
    dh = h64.abs() * 2.0 ** -20
    h = h64.bfloat16()
    loose = (h64 - dh).bfloat16() != (h64 + dh).bfloat16()
    assert loose.double().mean() < 0.01
    q, s = quantize_ref(h.float().cpu().numpy())
    q, s = torch.from_numpy(q.astype(np.int8)).to(DEV), torch.from_numpy(s).to(DEV)
    ref = dev_linear(q, s, *down).double()
    hf = h.double().abs()
    moves = (loose & (hf >= 0.98 * hf.amax(1, keepdim=True))).any(1, keepdim=True)
    per = torch.where(moves, 1.01 + q.double().abs() * 2.0 ** -7, loose.double()) * s[:, None]
    bound = per @ (down[0].double().abs() * down[1][:, None]).t()
    bound = torch.where(loose.any(1, keepdim=True), bound + 2.0 ** -21 * (ref.abs() + bound),
                        torch.zeros_like(bound))
    y = native.int8_mlp(x, gate, up, down, x_scales=xs, out_dtype=torch.float32)
    over = (y.double() - ref).abs() - bound
    assert (over <= 0).all(), f"{(over > 0).sum().item()} outside, worst {over.max().item()}"
    assert torch.equal(native.int8_mlp(x, gate, up, down, x_scales=xs), y.to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(16, 33, 1216), (17, 70, 640), (9, 100, 1120), (31, 4096, 1600),
                                   (32, 4112, 1600), (32, 8192, 96), (17, 8193, 96), (32, 64, 17408),
                                   (1, 50, 9984), (1, 50, 10240), (1, 50, 20352), (1, 50, 20480),
                                   (4, 30, 5088), (4, 30, 5120), (24, 40, 131040)])
def test_linear_at_the_rules(M, N, K):
    """Either side of the rules: x quantised inside (in little, in more LDS, with
    a workgroup per CU) or by a launch; few rows or a batch."""
    test_linear(M, N, K)


@pytest.mark.parametrize("T,H,I", [(1, 17440, 64), (1, 64, 17440), (16, 1024, 32), (17, 2048, 96),
                                   (32, 96, 4128), (32, 1568, 160), (33, 160, 1568), (24, 32, 8224)])
def test_mlp_at_the_rules(T, H, I):
    test_mlp(T, H, I)


@pytest.mark.parametrize("M", [1, 6])
def test_large_weights_equal_their_parts(M):
    """Weights past the size from which they are loaded as used once: columns of
    y as with the rows of W alone."""
    H, I, part = 5120, 13056, 384
    say("large weights", M)
    x = acts(M, H, 3).to(DEV)
    w, ws = dev_codes(2 * I, H, 5)
    y = native.int8_linear(x, w, ws)
    assert torch.equal(y[:, -part:], native.int8_linear(x, w[-part:].contiguous(),
                                                        ws[-part:].contiguous()))


@pytest.mark.parametrize("M", [1, 4, 5])
def test_long_weights_equal_their_parts(M):
    """As above, for the size from which up to 4 rows load them so."""
    N, K, part = 12832, 5120, 384
    say("long weights", M)
    x = acts(M, K, 3).to(DEV)
    w, ws = dev_codes(N, K, 5)
    y = native.int8_linear(x, w, ws)
    assert torch.equal(y[:, -part:], native.int8_linear(x, w[-part:].contiguous(),
                                                        ws[-part:].contiguous()))


# Products in two launches: (M, N, K, rows of x of a tile, rows of W, columns of
# y of the first launch); N odd, even and whole, K with every last block.
TWO_LAUNCHES = [(787, 19315, 928, 192, 256, 13056), (927, 16919, 288, 192, 256, 13056),
                (1425, 10922, 800, 192, 256, 8192), (1024, 17408, 1280, 256, 256, 16384),
                (984, 17388, 416, 256, 256, 16384)]
MLP_TWO_LAUNCHES = [(522, 13472, 288, 192, 256, 10880), (396, 16800, 1312, 256, 256, 16384)]


@pytest.mark.parametrize("M,N,K,rows,columns,main", TWO_LAUNCHES)
def test_linear_in_two_launches(M, N, K, rows, columns, main):
    say("two launches", M, N, K)
    assert native.int8_debug_plan(M, N, K) == (rows, columns, 1, main)
    (x, xs), (w, ws) = dev_codes(M, K, M), dev_codes(N, K, N)
    ref = dev_linear(x, xs, w, ws)
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full(((M + rows) * N,), 7.0, dtype=dt, device=DEV)
        out = buf[:M * N].view(M, N)
        native.int8_linear(x, w, ws, x_scales=xs, out=out)
        assert torch.equal(out, ref.to(dt)) and torch.all(buf[M * N:] == 7.0)


@pytest.mark.parametrize("T,I,H,rows,columns,main", MLP_TWO_LAUNCHES)
def test_mlp_in_two_launches(T, I, H, rows, columns, main):
    """The columns of h of either launch, seen through a down projection that
    keeps them: y as with the gate and up rows of one launch alone."""
    say("mlp two launches", T, I, H)
    assert native.int8_debug_plan(T, I, H, gate_up=True) == (rows, columns, 1, main)
    x, xs = dev_codes(T, H, T)
    gate, up = (dev_codes(I, H, s, 20.0 / H ** 0.5) for s in (1, 2))
    xs = xs * 100
    g, u = dev_linear(x, xs, *gate).double(), dev_linear(x, xs, *up).double()
    h64 = g / (1 + torch.exp(-g)) * u
    lo, hi = ((h64 - d * h64.abs() * 2.0 ** -20).bfloat16() for d in (1, -1))
    h = h64.bfloat16()
    top = h.float().abs().amax(1, keepdim=True)
    # identity rows of a down projection: y[t][j] = code of h[t][j] times the scale
    at = torch.randperm(I, generator=_gen(3))[:H].sort()[0].to(DEV)
    down = torch.zeros((H, I), dtype=torch.int8, device=DEV)
    down[torch.arange(H, device=DEV), at] = 1
    y = native.int8_mlp(x, gate, up, (down, torch.ones(H, device=DEV)), x_scales=xs,
                        out_dtype=torch.float32)
    # one code of the row's scale (and 2^-7 of it where the maximum may move), fp32 steps
    step = top / 127 * (0.5 + 2.0 ** -6) + h[:, at].float().abs() * 2.0 ** -7
    assert ((y - h[:, at].float()).abs() <= step).all()
    sure = (lo == hi).all(1)                  # rows whose h expf does not decide: exact
    q, s = quantize_ref(h.float().cpu().numpy())
    want = torch.from_numpy((q.astype(F32) * s[:, None]).astype(F32)).to(DEV)[:, at]
    assert torch.equal(y[sure], want[sure])


@pytest.mark.parametrize("M", [4, 5, 8, 9, 16, 17, 24, 25, 32])
@pytest.mark.parametrize("N", [4096, 4112, 4128, 5000, 6144, 6145])
def test_linear_of_two_row_tiles(M, N):
    """Codes given: 16 or 32 weight rows a workgroup, each number of groups of 8
    rows of x, odd last tiles."""
    test_linear(M, N, 416)


@pytest.mark.parametrize("M,N,K", [(1, 4112, 10080), (1, 4112, 10208), (15, 4112, 640),
                                   (16, 4112, 608), (17, 4112, 96), (2, 8192, 10112),
                                   (2, 8192, 10240), (2, 8208, 10112), (1, 13600, 10112),
                                   (1, 12800, 10112), (3, 4096, 10752), (3, 4096, 10880),
                                   (32, 4096, 992), (32, 4096, 1056)])
def test_where_x_is_quantised(M, N, K):
    """Either side of the rules by which a product quantises x itself: the bits
    of the product on the quantiser's codes, for gate and up as well."""
    say("quantised inside", M, N, K)
    x = acts(M, K, 7).to(DEV)
    q, s = native.int8_quantize(x)
    w, ws = dev_codes(N, K, N)
    for dt in (torch.float32, torch.bfloat16):
        y = native.int8_linear(x, w, ws, out_dtype=dt)
        assert torch.equal(y, dev_linear(q, s, w, ws).to(dt))
    N = N // 32 * 32
    mats = (w[:N], ws[:N].contiguous()), dev_codes(N, K, 2), dev_codes(K, N, 3)
    assert torch.equal(native.int8_mlp(x, *mats), native.int8_mlp(q, *mats, x_scales=s))


# Products with more than 2^31 bytes of codes of x, of W, or elements of y; the
# rows and columns at their ends, where an offset of 32 bits would be another.
LONG = [(70000, 80, 33024), (100, 70000, 33024), (70000, 33000, 64), (16, 70000, 33024)]


@pytest.mark.parametrize("M,N,K", LONG)
def test_linear_past_32_bits(M, N, K):
    say("long", M, N, K)
    g = torch.Generator(device=DEV).manual_seed(M)
    x, w = (torch.randint(-128, 128, (r, K), generator=g, dtype=torch.int8, device=DEV)
            for r in (M, N))
    xs, ws = (torch.rand(r, generator=g, device=DEV) * 1e-3 + 1e-4 for r in (M, N))
    y = native.int8_linear(x, w, ws, x_scales=xs)
    m, n = max(0, M - 24), max(0, N - 96)
    for r, c in ((slice(m, M), slice(n, N)), (slice(0, 24), slice(n, N)),
                 (slice(m, M), slice(0, 96))):
        part = native.int8_linear(x[r], w[c], ws[c].clone(), x_scales=xs[r].clone())
        assert torch.equal(y[r, c], part)
        ref = linear_ref(x[r].cpu().numpy(), xs[r].cpu().numpy(), w[c].cpu().numpy(),
                         ws[c].cpu().numpy())
        same(part, ref, (r, c))


@pytest.mark.parametrize("rows,cols", [(140000, 16384), (65600, 33024)])
def test_quantize_past_32_bits(rows, cols):
    say("long quantise", rows, cols)
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    q, s = native.int8_quantize(x)
    for r in (slice(0, 5), slice(rows // 2, rows // 2 + 5), slice(rows - 5, rows)):
        ref, top = quantize_ref(x[r].float().cpu().numpy())
        assert torch.equal(q[r].cpu().long(), torch.from_numpy(ref))
        assert torch.equal(s[r].cpu(), torch.from_numpy(top))
