"""The bf16 roundings of the RMS norm and of the int8 products at their ends:
subnormal results, ties, and sums that overflow."""
import numpy as np
import pytest
import torch

from nvfp4_routed_expert_amd import native
from test_gpu_int8 import DEV, codes, linear_ref, same, say
from test_gpu_norm import BF, FP, norm_ref

pytestmark = pytest.mark.gpu


def spread(rows, cols, seed, low, high):
    """fp32 values of every magnitude 2^low .. 2^high, some exact ties of bf16."""
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(low, high, (rows, cols), generator=g).float()
    m = 1 + torch.rand(rows, cols, generator=g)
    m = torch.where(torch.rand(rows, cols, generator=g) < 0.3,
                    1 + (2 * torch.randint(0, 128, (rows, cols), generator=g) + 1) / 256.0, m)
    sign = torch.randint(0, 2, (rows, cols), generator=g) * 2.0 - 1
    return (sign * m.double() * torch.exp2(e.double())).float()


@pytest.mark.parametrize("H", [96, 1056, 40960])
def test_norm(H):
    T = 6
    say("bf16 roundings, norm", H)
    x = spread(T, H, H, -149, -100)
    x[1] = spread(1, H, 2, -20, 10)[0]
    res = spread(T, H, H + 1, -149, -100).to(BF)
    res[2] = 0.0
    w = spread(1, H, 3, -140, 3)[0]
    n, total = norm_ref(x, w, res, eps=2.0 ** -40)
    for c in ("int8", "fp8", None):
        r = native.rms_norm_quantize(x.to(DEV), w.to(DEV), residual=res.to(DEV), eps=2.0 ** -40,
                                     codes=c, y_dtype=BF)
        assert torch.equal(r.residual.cpu().view(torch.int16), total.view(torch.int16))
        assert torch.equal(r.y.cpu(), torch.from_numpy(n).to(BF))


@pytest.mark.parametrize("H", [96, 40960])
def test_sum_that_overflows_bf16(H):
    """The sum of two finite numbers past bf16's largest is an infinity there."""
    say("bf16 overflow", H)
    x = torch.full((2, H), 1.0)
    res = torch.full((2, H), 1.0, dtype=BF)
    x[1, 5] = res[1, 5] = torch.finfo(BF).max
    w = torch.ones(H)
    r = native.rms_norm_quantize(x.to(DEV), w.to(DEV), residual=res.to(DEV), codes="int8")
    assert torch.equal(r.residual.cpu(), (x + res.float()).to(BF))
    assert torch.isinf(r.residual[1, 5]) and not torch.isfinite(r.scales[1])
    assert torch.isfinite(r.scales[0])


# few rows; a batch; a batch in K parts, with whole and with ragged rows of y
@pytest.mark.parametrize("M,N,K", [(3, 300, 512), (300, 500, 288), (40, 300, 8224), (40, 301, 8224)])
def test_products(M, N, K):
    say("bf16 roundings, linear", M, N, K)
    (x, xs), (w, ws) = codes(M, K, 1), codes(N, K, 2)
    xs = spread(1, M, 3, -126, -90)[0].abs()
    ws = spread(1, N, 4, -60, -20)[0].abs()
    ref = linear_ref(x.numpy(), xs.numpy(), w.numpy(), ws.numpy())
    tiny = np.abs(ref) < 2.0 ** -126
    assert 0.05 < tiny.mean() < 0.95
    same(native.int8_linear(x.to(DEV), w.to(DEV), ws.to(DEV), x_scales=xs.to(DEV)), ref, "bf16")
