"""RMS norm with the residual's addition and 8-bit outputs, bit for bit against
its definition: sums in 64 bits, every later step one fp32 operation."""
import sys

import numpy as np
import pytest
import torch

from nvfp4_routed_expert_amd import native
from test_gpu_fp8 import e4m3_table, quantize_ref as fp8_ref
from test_gpu_int8 import acts, quantize_ref as int8_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = np.float32
BF, FP = torch.bfloat16, torch.float32


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def norm_ref(x, w, res=None, eps=1e-6):
    """(n fp32, sum tensor or None) of torch tensors on the host."""
    total = None
    v = x.float()
    if res is not None:
        total = (v + res.float()).to(res.dtype)
        v = total.float()
    v = v.numpy()
    r = (1.0 / np.sqrt((v.astype(np.float64) ** 2).sum(1) / v.shape[1] + eps)).astype(F32)
    return ((v * r[:, None]).astype(F32) * w.float().numpy()[None]).astype(F32), total


def check(out, n, total, codes, y_dtype):
    if total is None:
        assert out.residual is None
    else:
        assert torch.equal(out.residual.cpu(), total)
    if y_dtype is None:
        assert out.y is None
    else:
        assert torch.equal(out.y.cpu(), torch.from_numpy(n).to(y_dtype))
    if codes == "int8":
        q, s = int8_ref(n)
        assert np.array_equal(out.scales.cpu().numpy(), s)
        assert np.array_equal(out.codes.cpu().numpy(), q)
    elif codes == "fp8":
        q, s = fp8_ref(n, 1)
        assert np.array_equal(out.scales.cpu().numpy(), s)
        assert np.array_equal(e4m3_table()[out.codes.cpu().numpy()], q)
    else:
        assert out.codes is None and out.scales is None


KINDS = [(BF, None, BF), (BF, BF, BF), (BF, FP, FP), (FP, None, BF), (FP, BF, FP), (FP, FP, BF)]
OUTS = [("fp8", None), ("int8", None), (None, BF), (None, FP), ("fp8", BF), ("int8", FP)]


@pytest.mark.parametrize("T,H", [(1, 32), (1, 5120), (3, 160), (17, 96), (5, 512), (5, 544),
                                 (9, 1024), (3, 1056), (66, 2048), (2, 8192), (2, 8224),
                                 (2, 16416), (2, 32768), (2, 32800), (1, 70016), (300, 64)])
@pytest.mark.parametrize("codes,y_dtype", OUTS)
def test_norm(T, H, codes, y_dtype):
    for i, (xt, rt, wt) in enumerate(KINDS):
        say("norm", T, H, codes, y_dtype, xt, rt)
        x, w = acts(T, H, T + H, xt), acts(1, H, H, wt)[0]
        res = None if rt is None else acts(T, H, T + H + 1, rt)
        out = native.rms_norm_quantize(x.to(DEV), w.to(DEV),
                                       residual=None if res is None else res.to(DEV),
                                       codes=codes, y_dtype=y_dtype)
        check(out, *norm_ref(x, w, res), codes, y_dtype)


def test_rows_of_zeros_small_and_large():
    """A zero row (r is 1 / sqrt(eps)), one that the residual cancels, one of
    subnormals, one whose squares pass 32 bits, one large element; eps at its
    bounds."""
    H = 544
    x, res = acts(8, H, 1, FP), acts(8, H, 2, FP)
    x[0] = res[0] = 0.0
    x[1] = -res[1]
    x[2] = res[2] = 1e-40
    x[3] = res[3] = 1e38
    x[4, 100], res[4] = 3e4, 0.0
    x[5] = res[5] = 0.0
    x[5, 500] = 1.0
    w = acts(1, H, 3, FP)[0]
    w[7] = 0.0
    w[9] = -w[9]
    for eps in (1e-6, 2.0 ** -126, 1.0, 2.0 ** 125):
        for codes in ("int8", "fp8"):
            say("extremes", eps, codes)
            out = native.rms_norm_quantize(x.to(DEV), w.to(DEV), residual=res.to(DEV), eps=eps,
                                           codes=codes, y_dtype=FP)
            check(out, *norm_ref(x, w, res, eps), codes, FP)


@pytest.mark.parametrize("H", [96, 1056, 5120, 40960])
def test_strides_and_in_place(H):
    """Strided rows of x and of the residual; the sum over the residual, over x
    (same type), or into a strided place of its own, whose other columns and
    rows are left."""
    T = 7
    say("strides", H)
    w = acts(1, H, 3)[0]
    wide = acts(T, 2 * H + 64, 5, BF)
    x, res = wide[:, :H], wide[:, H + 32: 2 * H + 32]
    n, total = norm_ref(x, w, res)
    d = wide.to(DEV)
    xd, rd = d[:, :H], d[:, H + 32: 2 * H + 32]
    buf = torch.full((T + 2, H + 64), 7.0, dtype=BF, device=DEV)
    place = buf[1:T + 1, 32:H + 32]
    out = native.rms_norm_quantize(xd, w.to(DEV), residual=rd, codes="int8", y_dtype=BF,
                                   out=native.RmsNorm(None, None, None, place))
    check(out, n, total, "int8", BF)
    assert torch.equal(d.cpu(), wide)
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert (buf[:, :32] == 7).all() and (buf[:, H + 32:] == 7).all()
    for where in ("residual", "x"):
        xc, rc = x.clone().to(DEV), res.clone().to(DEV)
        to = rc if where == "residual" else xc
        out = native.rms_norm_quantize(xc, w.to(DEV), residual=rc, codes="fp8", y_dtype=FP,
                                       out=native.RmsNorm(None, None, None, to))
        assert out.residual is to
        check(out, n, total, "fp8", FP)
        assert torch.equal((xc if where == "residual" else rc).cpu(),
                           x if where == "residual" else res)


def test_given_outputs_and_their_neighbours():
    T, H = 5, 288
    say("given outputs")
    x, w = acts(T, H, 1), acts(1, H, 2)[0]
    n, _ = norm_ref(x, w)
    for codes, t, cols in (("int8", torch.int8, 1), ("fp8", torch.uint8, 3)):
        q = torch.full((T + 2, H), 7, dtype=t, device=DEV)
        s = torch.full((T + 8, cols), 7.0, device=DEV)
        y = torch.full((T + 2, H), 7.0, dtype=FP, device=DEV)
        sv = s[4:4 + T] if codes == "fp8" else s[4:4 + T, 0]
        o = native.RmsNorm(y[1:T + 1], q[1:T + 1], sv, None)
        got = native.rms_norm_quantize(x.to(DEV), w.to(DEV), codes=codes, y_dtype=FP, out=o)
        check(got, n, None, codes, FP)
        assert (q[0] == 7).all() and (q[-1] == 7).all() and (y[0] == 7).all() and (y[-1] == 7).all()
        assert (s[:4] == 7).all() and (s[4 + T:] == 7).all()


def test_empty_batch():
    x, w = torch.empty((0, 96), dtype=BF, device=DEV), torch.ones(96, device=DEV)
    out = native.rms_norm_quantize(x, w, residual=x, codes="fp8", y_dtype=BF)
    assert out.y.shape == (0, 96) and out.codes.shape == (0, 96) and out.scales.shape == (0, 1)


def test_binding_refuses_other_shapes_and_devices():
    x, w = acts(3, 96, 1).to(DEV), torch.ones(96, device=DEV)
    call = lambda *a, **k: native.rms_norm_quantize(*a, codes="int8", **k)
    with pytest.raises(ValueError, match="weight has shape"):
        call(x, w[:64])
    with pytest.raises(ValueError, match="weight is on"):
        call(x, w.cpu())
    with pytest.raises(ValueError, match="residual is on"):
        call(x, w, residual=x.cpu())
    with pytest.raises(ValueError, match="residual has shape"):
        call(x, w, residual=x[:2])
    with pytest.raises(TypeError, match="unsupported dtype"):
        call(x.half(), w)
    with pytest.raises(TypeError, match="codes is"):
        call(x, w, out=native.RmsNorm(None, torch.empty((3, 96), dtype=torch.uint8, device=DEV),
                                      None, None))
    with pytest.raises(native.NVFP4Error, match="overlaps"):
        call(x, w, y_dtype=BF, out=native.RmsNorm(x, None, None, None))
    with pytest.raises(native.NVFP4Error, match="eps"):
        call(x, w, eps=0.0)


def test_norm_in_a_graph():
    T, H = 9, 1056
    say("graph")
    w = acts(1, H, 2)[0].to(DEV)
    x, res = acts(T, H, 1).to(DEV), acts(T, H, 3).to(DEV)
    out = native.rms_norm_quantize(x, w, residual=res, codes="int8", y_dtype=BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        native.rms_norm_quantize(x, w, residual=res, codes="int8", y_dtype=BF, out=out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.rms_norm_quantize(x, w, residual=res, codes="int8", y_dtype=BF, out=out)
    for seed in range(4):
        x.copy_(acts(T, H, 40 + seed))
        want = native.rms_norm_quantize(x, w, residual=res, codes="int8", y_dtype=BF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("T,H", [(140000, 16384), (65600, 33024)])
@pytest.mark.parametrize("codes", ["int8", "fp8"])
def test_norm_past_32_bits(T, H, codes):
    """More than 2^31 elements: the first, middle and last rows."""
    say("long norm", T, H, codes)
    g = torch.Generator(device=DEV).manual_seed(T)
    x, res = (torch.empty((T, H), dtype=BF, device=DEV).normal_(generator=g) for _ in range(2))
    w = acts(1, H, H)[0]
    rows = [slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)]
    was = [(x[r].cpu(), res[r].cpu()) for r in rows]
    out = native.rms_norm_quantize(x, w.to(DEV), residual=res, codes=codes, y_dtype=BF,
                                   out=native.RmsNorm(None, None, None, res))
    for r, (a, b) in zip(rows, was):
        check(native.RmsNorm(*(t[r] for t in out)), *norm_ref(a, w, b), codes, BF)
