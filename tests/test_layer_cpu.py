"""Refusals of moe_layer_decode: the documented status before anything is
enqueued (C ABI), and the binding's checks (no GPU needed)."""
import ctypes
import os

import pytest
import torch

from nvfp4_routed_expert_amd import native, weights

pytestmark = pytest.mark.skipif(not os.path.exists(native.LIB_PATH),
                                reason="library not built")

FAKE, MIS = 1 << 20, (1 << 20) + 4          # never dereferenced


def _last():
    return native.lib().nvfp4_last_error().decode()


def make(H=256, I=64, E=8, k=2, router=FAKE, bias=None, experts=None, Is=32, sg=FAKE, su=FAKE,
         sd=FAKE, gate=None):
    w = native.ExpertWeightsC(*(experts or [FAKE] * 9))
    return native.MoeLayerC(H, I, E, k, router, bias, w, Is, sg, su, sd, gate)


def call(layer, T=4, x=FAKE, ids=FAKE, wts=FAKE, y=FAKE, dt=0, ws=FAKE, nbytes=1 << 26):
    v = lambda p: None if p is None else ctypes.c_void_p(p)
    return native.lib().moe_layer_decode(v(x), T, None if layer is None else ctypes.byref(layer), 1,
                                         v(ids), v(wts), v(y), dt, v(ws), nbytes, None)


def test_null_and_misaligned_pointers():
    for kw in ("x", "ids", "wts", "y"):
        assert call(make(), **{kw: None}) == 1, kw
        assert call(make(), **{kw: MIS}) == 3, kw
    assert call(None) == 1
    assert call(make(router=None)) == 1 and call(make(router=MIS)) == 3
    assert call(make(bias=MIS)) == 3 and call(make(gate=MIS)) == 3
    for i in range(9):
        bad = [FAKE] * 9
        bad[i] = None
        assert call(make(experts=bad)) == 1
        bad[i] = MIS if i < 6 else FAKE + 2
        assert call(make(experts=bad)) == 3
    for kw in ("sg", "su", "sd"):
        assert call(make(**{kw: None})) == 1 and "shared" in _last()
        assert call(make(**{kw: MIS})) == 3


def test_sizes():
    assert call(make(), T=-1) == 1
    assert call(make(), T=65) == 2 and "64 tokens" in _last()
    assert call(make(E=32, k=16), T=33) == 2          # T * k > 512
    assert call(make(k=0)) == 2 and call(make(k=9)) == 2 and call(make(E=64, k=33)) == 2
    assert call(make(E=0)) == 2 and call(make(E=1025)) == 2
    assert call(make(H=48)) == 2 and call(make(I=80)) == 2 and call(make(Is=40)) == 2
    assert call(make(H=0)) == 2 and call(make(Is=-32)) == 1
    assert call(make(H=(1 << 13) + 32)) == 2 and call(make(I=(1 << 20) + 32)) == 2
    assert call(make(H=1 << 13, I=(1 << 19) + 32)) == 2 and "2^32" in _last()
    assert call(make(), dt=3) == 1
    assert call(make(Is=0, sg=None, su=None, sd=None, gate=FAKE)) == 1


def test_workspace():
    L = native.lib()
    n = L.moe_layer_decode_workspace_size(4, 256, 64, 8, 2, 32)
    assert n >= 4 * 2 * 256 * 4
    assert call(make(), nbytes=n - 1) == 4 and "workspace" in _last()
    assert call(make(), ws=None, nbytes=n) == 1
    assert call(make(), ws=MIS, nbytes=n) == 3
    assert L.moe_layer_decode_workspace_size(0, 256, 64, 8, 2, 32) == 0


def test_empty_batch_checks_the_layer():
    assert call(make(), T=0, x=None, ids=None, wts=None, y=None, ws=None, nbytes=0) == 0
    assert call(make(H=48), T=0, x=None, ids=None, wts=None, y=None, ws=None, nbytes=0) == 2


def test_binding_refusals():
    w = weights.empty_experts(4, 64, 32, "cpu")
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    r = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cuda"):
        native.moe_layer_decode(x, r, w, 2)
    with pytest.raises(TypeError, match="bfloat16"):
        native.moe_layer_decode(x.float(), r, w, 2)
    with pytest.raises(ValueError, match="router_w"):
        native.moe_layer_decode(x, r[:3], w, 2)
    with pytest.raises(ValueError, match="hidden"):
        native.moe_layer_decode(x[:, :32], r[:, :32], w, 2)
    with pytest.raises(ValueError, match="bias"):
        native.moe_layer_decode(x, r, w, 2, bias=torch.zeros(3))
    with pytest.raises(ValueError, match="shared_gate"):
        native.moe_layer_decode(x, r, w, 2, shared_gate=x[0])
    s = torch.zeros((32, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shared down"):
        native.moe_layer_decode(x, r, w, 2, shared=(s, s, s))


@pytest.mark.parametrize("n", [0, 1, 2, 4])
def test_shared_expert_is_three_matrices(n):
    """With two of them and a shared gate, the gate's [H] vector would be taken
    for the [H, shared_I] down projection and read past its end."""
    w = weights.empty_experts(4, 64, 32, "cpu")
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    r = torch.zeros((4, 64), dtype=torch.bfloat16)
    s, d = torch.zeros((32, 64), dtype=torch.bfloat16), torch.zeros((64, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shared must be"):
        native.moe_layer_decode(x, r, w, 2, shared=(s, s, d, d)[:n], shared_gate=x[0])


@pytest.mark.parametrize("H,I,E,k,Is", [(2048, 512, 512, 8, 512), (4096, 1536, 128, 8, 0),
                                        (256, 2080, 6, 2, 32), (1024, 8192, 64, 1, 0),
                                        (512, 96, 1024, 32, 544)])
def test_workspace_of_a_batch_serves_smaller_ones(H, I, E, k, Is):
    """A decode loop allocates once, for its largest batch: also where fewer
    tokens take narrower slices, and so more partial rows each."""
    size = native.lib().moe_layer_decode_workspace_size
    sizes = [size(T, H, I, E, k, Is) for T in range(65)]
    assert sizes == sorted(sizes) and sizes[1] > 0


def test_the_gpu_tests_reach_every_kernel():
    """The rule that picks a kernel is host code: a changed one shows here, before
    the GPU tests lose what they are for."""
    import test_gpu_layer as g
    reached = set()
    cases = [c for c, _ in g.KERNEL_CASES]
    for f in (g.test_layer, g.test_layer_of_crowded_experts, g.test_layer_of_large_experts):
        for m in f.pytestmark:
            if m.name == "parametrize":
                cases += m.args[1]
    for T, H, I, E, k, *_ in cases:
        cols, tokens, once = native.layer_debug_plan(T, H, I, E, k)
        reached.add((cols, H % 128 == 0 and I % 128 == 0, tokens, once))
    assert reached == {(c, a, t, o) for c in (128, 256) for a in (False, True)
                       for t in (1, 2, 4) for o in (False, True)}
    for (T, H, I, E, k, *_), plan in g.KERNEL_CASES:
        cols, tokens, once = native.layer_debug_plan(T, H, I, E, k)
        assert (cols, H % 128 == 0 and I % 128 == 0, tokens, once) == plan


def test_workspace_of_a_batch_that_is_refused():
    """A batch past the call's limits is not made to allocate for its size before
    it is refused: the query answers for the largest one that is not."""
    size = native.lib().moe_layer_decode_workspace_size
    assert size(1 << 16, 4096, 1536, 128, 8, 0) == size(64, 4096, 1536, 128, 8, 0)
    assert size(65, 256, 64, 64, 32, 32) == size(16, 256, 64, 64, 32, 32)
    assert size(1 << 40, 256, 64, 8, 2, 32) == size(64, 256, 64, 8, 2, 32)
