"""A NaN or an infinity in a row of the int8 quantiser, of the RMS norm and of the
int8 products: the row's scale, and every product of the row, is not finite, and
the other rows are those of the batch without it, bit for bit."""
import sys

import pytest
import torch

from nvfp4_routed_expert_amd import native
from test_gpu_int8 import acts, codes

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32
BAD = [float("nan"), float("inf"), float("-inf")]


def say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


def rows_with(x, bad):
    """x with `bad` in one element of each of some rows, and those rows."""
    T, H = x.shape
    places = {0: 0, T // 2: H // 2 + 3, T - 1: H - 1}
    y = x.clone()
    for row, col in places.items():
        y[row, col] = bad
    hit = torch.zeros(T, dtype=torch.bool)
    hit[list(places)] = True
    return y, hit


# 1 to 16 waves a row, and rows past 32768 columns
@pytest.mark.parametrize("T,H", [(1, 32), (9, 96), (7, 1056), (2100, 1056), (5, 5120), (1200, 5120),
                                 (5, 17408), (6, 40960)])
@pytest.mark.parametrize("bad", BAD)
def test_quantize(T, H, bad):
    for dtype in (BF, FP):
        say("quantize", T, H, bad, dtype)
        x = acts(T, H, T + H, dtype)
        y, hit = rows_with(x, bad)
        q, s = (t.cpu() for t in native.int8_quantize(y.to(DEV)))
        q0, s0 = (t.cpu() for t in native.int8_quantize(x.to(DEV)))
        assert not torch.isfinite(s[hit]).any()
        assert torch.equal(s[~hit], s0[~hit]) and torch.equal(q[~hit], q0[~hit])


@pytest.mark.parametrize("T,H", [(1, 32), (9, 96), (7, 1056), (2100, 1056), (5, 5120), (1200, 5120),
                                 (5, 17408), (6, 40960)])
@pytest.mark.parametrize("bad", BAD)
def test_norm_int8(T, H, bad):
    w = acts(1, H, 3)[0].to(DEV)
    for res_type in (None, BF):
        say("norm", T, H, bad, res_type)
        x = acts(T, H, T + H)
        res = None if res_type is None else acts(T, H, T + 1, res_type).to(DEV)
        y, hit = rows_with(x, bad)
        r = native.rms_norm_quantize(y.to(DEV), w, residual=res, codes="int8", y_dtype=BF)
        r0 = native.rms_norm_quantize(x.to(DEV), w, residual=res, codes="int8", y_dtype=BF)
        s, s0 = r.scales.cpu(), r0.scales.cpu()
        assert not torch.isfinite(s[hit]).any()
        assert torch.equal(s[~hit], s0[~hit])
        assert torch.equal(r.codes.cpu()[~hit], r0.codes.cpu()[~hit])
        assert torch.equal(r.y.cpu()[~hit], r0.y.cpu()[~hit])


# few rows quantised inside (1 to 32 rows, rows of one and of several pieces), few
# rows and batches behind a quantiser of their own
@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (2, 64, 96), (3, 300, 2080), (16, 1000, 544),
                                   (31, 70, 640), (16, 2048, 2016), (8, 4200, 8224),
                                   (4, 4200, 640), (40, 300, 1056), (300, 500, 288)])
@pytest.mark.parametrize("bad", BAD)
def test_linear(M, N, K, bad):
    say("linear", M, N, K, bad)
    x = acts(M, K, M * 7 + K)
    y, hit = rows_with(x, bad)
    w, ws = (t.to(DEV) for t in codes(N, K, N + K))
    want = native.int8_linear(x.to(DEV), w, ws).cpu()
    got = native.int8_linear(y.to(DEV), w, ws).cpu()
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[~hit], want[~hit])
    q, s = native.int8_quantize(y.to(DEV))
    parts = native.int8_linear(q, w, ws, x_scales=s).cpu()
    assert torch.equal(got.view(torch.int16)[~hit], parts.view(torch.int16)[~hit])
    assert torch.equal(torch.isnan(got), torch.isnan(parts))
    assert torch.equal(got.nan_to_num(nan=0.0), parts.nan_to_num(nan=0.0))


@pytest.mark.parametrize("T,H,I", [(1, 512, 1056), (3, 2080, 320), (16, 96, 2048), (40, 288, 160),
                                   (300, 160, 288)])
@pytest.mark.parametrize("bad", BAD)
def test_mlp(T, H, I, bad):
    say("mlp", T, H, I, bad)
    x = acts(T, H, T * 7 + H)
    y, hit = rows_with(x, bad)
    gate, up, down = ([t.to(DEV) for t in codes(n, k, n + k + s)]
                      for n, k, s in ((I, H, 0), (I, H, 1), (H, I, 2)))
    want = native.int8_mlp(x.to(DEV), gate, up, down).cpu()
    got = native.int8_mlp(y.to(DEV), gate, up, down).cpu()
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("T,H", [(1, 32), (9, 96), (7, 1056), (2100, 1056), (5, 5120), (1200, 5120),
                                 (5, 17408), (6, 40960)])
@pytest.mark.parametrize("bad", BAD)
def test_norm_fp8(T, H, bad):
    """The scale of the 128 columns that hold it (a NaN: of all of the row's)."""
    w = acts(1, H, 3)[0].to(DEV)
    say("norm fp8", T, H, bad)
    x = acts(T, H, T + H)
    y, hit = rows_with(x, bad)
    r = native.rms_norm_quantize(y.to(DEV), w, codes="fp8")
    r0 = native.rms_norm_quantize(x.to(DEV), w, codes="fp8")
    s, s0 = r.scales.cpu(), r0.scales.cpu()
    pad = torch.nn.functional.pad(y.float(), (0, -H % 128)).view(T, -1, 128)
    blocks = ~torch.isfinite(pad).all(2) if bad == bad else hit[:, None].expand(T, s.shape[1])
    assert not torch.isfinite(s[blocks]).any()
    assert torch.equal(s[~hit], s0[~hit])
    assert torch.equal(r.codes.cpu()[~hit], r0.codes.cpu()[~hit])
    assert (r.codes.cpu() & 0x7F != 0x7F).all()


@pytest.mark.parametrize("T,H,N", [(1, 512, 300), (9, 1056, 96), (90, 2048, 500)])
@pytest.mark.parametrize("bad", BAD)
def test_norm_in_front_of_an_fp8_product(T, H, N, bad):
    say("norm, fp8 product", T, H, N, bad)
    x, w = acts(T, H, T + H), acts(1, H, 3)[0].to(DEV)
    y, hit = rows_with(x, bad)
    wq = native.fp8_block_quantize(acts(N, H, 5).to(DEV), 128)
    got, want = (native.fp8_block_linear(r.codes, *wq, x_scales=r.scales).cpu() for r in
                 (native.rms_norm_quantize(t.to(DEV), w, codes="fp8") for t in (y, x)))
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[~hit], want[~hit])


def all_ones(x, row, col):
    """x with a NaN of all ones at one element."""
    y = x.clone()
    y.view(torch.int32)[row, col] = -1
    assert torch.isnan(y[row, col])
    return y


@pytest.mark.parametrize("H", [96, 1056, 40960])
def test_nan_of_all_ones_in_the_norm(H):
    """Rounded to bf16 it stays NaN, in the sum and in y."""
    T = 5
    say("nan of all ones, norm", H)
    x, w = acts(T, H, 1, FP), acts(1, H, 2)[0].to(DEV)
    res = torch.zeros(T, H, dtype=BF)
    y = all_ones(x, 2, 7)
    for codes_ in ("int8", "fp8"):
        r = native.rms_norm_quantize(y.to(DEV), w, residual=res.to(DEV), codes=codes_, y_dtype=BF)
        assert torch.isnan(r.residual.cpu()[2, 7]) and torch.isnan(r.y.cpu()[2]).all()
        assert not torch.isfinite(r.scales.cpu()[2]).any()
        r0 = native.rms_norm_quantize(x.to(DEV), w, residual=res.to(DEV), codes=codes_, y_dtype=BF)
        rest = [0, 1, 3, 4]
        assert torch.equal(r.y.cpu()[rest], r0.y.cpu()[rest])
        assert torch.equal(r.residual.cpu()[rest], r0.residual.cpu()[rest])


# few rows; a batch; a batch in K parts, with rows of y that are not whole quads
@pytest.mark.parametrize("M,N,K", [(3, 300, 512), (300, 500, 288), (40, 301, 8224), (40, 300, 8224)])
def test_nan_of_all_ones_in_a_product(M, N, K):
    say("nan of all ones, linear", M, N, K)
    x = acts(M, K, 3, FP)
    q, s = native.int8_quantize(all_ones(x, M - 1, K - 1).to(DEV))
    w, ws = (t.to(DEV) for t in codes(N, K, N + K))
    for scale in (s, all_ones(s.cpu()[:, None], M - 1, 0)[:, 0].to(DEV)):
        y = native.int8_linear(q, w, ws, x_scales=scale).cpu()
        assert torch.isnan(y[M - 1]).all() and torch.isfinite(y[:M - 1]).all()
