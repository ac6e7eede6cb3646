"""More rows than one launch of the int8 quantiser and of the RMS norm has
workgroups for."""
import pytest
import torch

from nvfp4_routed_expert_amd import native
from test_gpu_int8 import acts, quantize_ref
from test_gpu_norm import BF, DEV, check, norm_ref, say

pytestmark = pytest.mark.gpu

# Past the largest launch (2^20 workgroups) a workgroup takes rows in turn: from
# 2^22 rows on with one wave a row, 2^21 with two, 2^20 with 4 and 16 waves and for
# rows past 32768 columns.
MANY_ROWS = [((1 << 22) + (1 << 20) + 5, 32), ((1 << 21) + (1 << 18) + 1, 2624),
             ((1 << 20) + (1 << 17) + 3, 5184), ((1 << 20) + (1 << 16) + 1, 20512),
             ((1 << 20) + (1 << 15) + 1, 32800)]


def many_rows(rows, cols):
    """Random bf16 rows of different magnitudes."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    for r in range(0, rows, 1 << 18):
        x[r:r + (1 << 18)].normal_(generator=g)
    return x.mul_(torch.rand((rows, 1), generator=g, device=DEV).bfloat16() + 0.5)


@pytest.mark.parametrize("rows,cols", MANY_ROWS)
def test_quantize_of_many_rows(rows, cols):
    """As the rows in calls that a launch holds, bit for bit, and some against the
    plain form."""
    say("quantise many rows", rows, cols)
    x = many_rows(rows, cols)
    q, s = native.int8_quantize(x)
    for r in range(0, rows, 1 << 19):
        part = native.int8_quantize(x[r:r + (1 << 19)])
        assert torch.equal(q[r:r + (1 << 19)], part[0]) and torch.equal(s[r:r + (1 << 19)], part[1])
    for r in (0, (1 << 20) - 2, (1 << 20) - 1, 1 << 20, rows - 3):
        ref, top = quantize_ref(x[r:r + 3].float().cpu().numpy())
        assert torch.equal(q[r:r + 3].cpu().long(), torch.from_numpy(ref))
        assert torch.equal(s[r:r + 3].cpu(), torch.from_numpy(top))


@pytest.mark.parametrize("T,H", MANY_ROWS)
@pytest.mark.parametrize("codes", ["int8", "fp8"])
def test_norm_of_many_rows(T, H, codes):
    """More rows than a launch has workgroups for: as the rows in smaller calls,
    bit for bit, and some against the plain form; to int8 also the sum with a
    residual, over x."""
    say("norm of many rows", T, H, codes)
    x, w = many_rows(T, H), acts(1, H, H)[0]
    wd = w.to(DEV)
    at = [(r, x[r:r + 3].cpu()) for r in (0, (1 << 20) - 2, 1 << 20, T - 3)]
    out = native.rms_norm_quantize(x, wd, codes=codes)
    for r in range(0, T, 1 << 19):
        part = native.rms_norm_quantize(x[r:r + (1 << 19)], wd, codes=codes)
        assert torch.equal(out.codes[r:r + (1 << 19)], part.codes)
        assert torch.equal(out.scales[r:r + (1 << 19)], part.scales)
    for r, was in at:
        check(native.RmsNorm(None, out.codes[r:r + 3], out.scales[r:r + 3], None),
              *norm_ref(was, w), codes, None)
    if codes == "fp8" or T * H > 1 << 33:
        return
    res = torch.roll(x, 1, 0)
    at = [(r, x[r:r + 3].cpu(), res[r:r + 3].cpu()) for r in (0, (1 << 20) - 2, 1 << 20, T - 3)]
    want = []
    for r in range(0, T, 1 << 19):
        part = native.rms_norm_quantize(x[r:r + (1 << 19)], wd, residual=res[r:r + (1 << 19)],
                                        codes="int8")
        want.append(part)
    out = native.rms_norm_quantize(x, wd, residual=res, codes="int8", y_dtype=BF,
                                   out=native.RmsNorm(None, None, None, x))
    for r, part in zip(range(0, T, 1 << 19), want):
        n = slice(r, r + (1 << 19))
        assert torch.equal(out.codes[n], part.codes) and torch.equal(out.scales[n], part.scales)
        assert torch.equal(x[n], part.residual)
    for r, a, b in at:
        check(native.RmsNorm(*(t[r:r + 3] for t in out)), *norm_ref(a, w, b), "int8", BF)
