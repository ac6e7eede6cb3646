"""The int8 operators and the RMS norm at the largest sizes that they take: 2^24
rows of x or of W, rows of 2^27 columns."""
import numpy as np
import pytest
import torch

from nvfp4_routed_expert_amd import native
from test_gpu_fp8 import e4m3_table, quantize_ref as fp8_ref
from test_gpu_int8 import acts, dev_codes, dev_linear, quantize_ref, say
from test_gpu_norm import norm_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32
MOST = 1 << 24


@pytest.mark.parametrize("M,N", [(1, MOST), (33, MOST), (MOST, 1), (MOST, 35)])
def test_linear(M, N):
    """Every output, against sums in 64 bits."""
    say("bounds linear", M, N)
    K, step = 32, 1 << 20
    (x, xs), (w, ws) = dev_codes(M, K, 1), dev_codes(N, K, 2)
    y = native.int8_linear(x, w, ws, x_scales=xs, out_dtype=FP)
    for m in range(0, M, step):
        for n in range(0, N, step):
            a, b = slice(m, m + step), slice(n, n + step)
            assert torch.equal(y[a, b], dev_linear(x[a], xs[a], w[b], ws[b]))


def test_mlp():
    """As the tokens in smaller batches, x quantised by the call."""
    say("bounds mlp")
    H, I, step = 32, 64, 1 << 22
    x = torch.empty((MOST, H), dtype=BF, device=DEV).normal_(
        generator=torch.Generator(device=DEV).manual_seed(1))
    mats = [dev_codes(n, k, s, 3.0) for s, (n, k) in ((1, (I, H)), (2, (I, H)), (3, (H, I)))]
    y = native.int8_mlp(x, *mats)
    assert torch.isfinite(y).all() and y.float().abs().amax() > 0
    for r in range(0, MOST, step):
        assert torch.equal(y[r:r + step], native.int8_mlp(x[r:r + step], *mats))
    assert torch.equal(y[-3:], native.int8_mlp(x[-3:], *mats))


def test_more_is_refused():
    w, ws = dev_codes(32, 32, 1)
    x = torch.zeros((MOST + 1, 32), dtype=BF, device=DEV)
    with pytest.raises(native.NVFP4Error, match="2\\^24"):
        native.int8_linear(x, w, ws)
    with pytest.raises(native.NVFP4Error, match="2\\^24"):
        native.int8_mlp(x, (w, ws), (w, ws), (w, ws))
    with pytest.raises(native.NVFP4Error, match="2\\^24"):
        native.int8_quantize(x)
    with pytest.raises(native.NVFP4Error, match="2\\^24"):
        native.rms_norm_quantize(x, torch.ones(32, device=DEV), codes="int8")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_longest_rows(dtype):
    """Two rows of 2^27 columns, and a last block of 32."""
    for H in (1 << 27, (1 << 27) - 96):
        say("bounds rows", H, dtype)
        g = torch.Generator(device=DEV).manual_seed(3)
        x = torch.empty((2, H), dtype=dtype, device=DEV).normal_(generator=g)
        q, s = native.int8_quantize(x)
        ref, top = quantize_ref(x.float().cpu().numpy())
        assert np.array_equal(s.cpu().numpy(), top)
        assert torch.equal(q.cpu().long(), torch.from_numpy(ref))


def test_norm_of_the_longest_row():
    H = (1 << 27) - 96
    say("bounds norm", H)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty((1, H), dtype=BF, device=DEV).normal_(generator=g)
    w = torch.rand(H, generator=g, device=DEV) + 0.5
    n, _ = norm_ref(x.cpu(), w.cpu())
    r = native.rms_norm_quantize(x, w, codes="int8", y_dtype=FP)
    q, s = quantize_ref(n)
    assert np.array_equal(r.y.cpu().numpy(), n) and np.array_equal(r.scales.cpu().numpy(), s)
    assert torch.equal(r.codes.cpu().long(), torch.from_numpy(q))
    f = native.rms_norm_quantize(x, w, codes="fp8")
    q, s = fp8_ref(n, 1)
    assert np.array_equal(f.scales.cpu().numpy(), s)
    assert np.array_equal(e4m3_table()[f.codes.cpu().numpy()], q)


def test_sum_over_x_and_of_x_with_itself():
    """The residual's sum over an f32 x, and x as its own residual, replaced."""
    for H in (1056, 40960):
        say("in place", H)
        w = acts(1, H, 3)[0]
        x, res = acts(5, H, 1, FP), acts(5, H, 2, FP)
        n, total = norm_ref(x, w, res)
        xd = x.to(DEV)
        out = native.rms_norm_quantize(xd, w.to(DEV), residual=res.to(DEV), codes="int8", y_dtype=FP,
                                       out=native.RmsNorm(None, None, None, xd))
        assert torch.equal(xd.cpu(), total) and np.array_equal(out.y.cpu().numpy(), n)
        n, total = norm_ref(x, w, x)
        xd = x.to(DEV)
        out = native.rms_norm_quantize(xd, w.to(DEV), residual=xd, codes="int8", y_dtype=FP,
                                       out=native.RmsNorm(None, None, None, xd))
        assert torch.equal(xd.cpu(), total) and np.array_equal(out.y.cpu().numpy(), n)
