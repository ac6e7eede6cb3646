"""The gated int8 MLP of a few tokens with weights that are loaded as used once."""
import numpy as np
import pytest
import torch

from nvfp4_routed_expert_amd import native
from test_gpu_int8 import dev_codes, mlp_ref, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mats():
    """Gate and up past the size from which they are loaded so (128 MB)."""
    H, I = 5120, 12832
    return [dev_codes(n, k, s, 20.0 / k ** 0.5)
            for s, (n, k) in ((1, (I, H)), (2, (I, H)), (3, (H, I)))]


def tokens(T, H):
    x, xs = dev_codes(T, H, T)
    return x, xs * 100


@pytest.mark.parametrize("T", [3, 5, 8, 9, 16, 17, 24, 25, 32])
def test_few_tokens_as_in_a_batch(mats, T):
    """Codes given, each number of groups of 8 tokens: the bits of the same tokens
    in a batch of 64, which takes another form."""
    say("streamed mlp", T)
    H, I = mats[2][0].shape
    assert native.int8_debug_plan(T, I, H, gate_up=True)[0] == 0
    assert native.int8_debug_plan(64, I, H, gate_up=True)[0] == 64
    x, xs = tokens(64, H)
    for dt in (torch.float32, torch.bfloat16):
        y = native.int8_mlp(x[:T], *mats, x_scales=xs[:T], out_dtype=dt)
        assert torch.equal(y, native.int8_mlp(x, *mats, x_scales=xs, out_dtype=dt)[:T])


@pytest.mark.parametrize("T", [6, 26])
def test_few_tokens_against_the_plain_form(mats, T):
    say("streamed mlp, plain form", T)
    x, xs = tokens(T, mats[2][0].shape[0])
    ref, bound, loose = mlp_ref(x.cpu().numpy(), xs.cpu().numpy(),
                                *[tuple(t.cpu().numpy() for t in m) for m in mats])
    assert loose.mean() < 0.01
    y = native.int8_mlp(x, *mats, x_scales=xs, out_dtype=torch.float32)
    over = np.abs(y.double().cpu().numpy() - ref) - bound
    assert (over <= 0).all(), f"{(over > 0).sum()} outside, worst {over.max()}"
