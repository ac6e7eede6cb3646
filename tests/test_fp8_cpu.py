"""Refusals of the FP8 block-scaled entry points: the documented status before
anything is enqueued (C ABI), and the binding's checks (no GPU needed)."""
import ctypes
import os

import pytest
import torch

from nvfp4_routed_expert_amd import native

pytestmark = pytest.mark.skipif(not os.path.exists(native.LIB_PATH),
                                reason="library not built")

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 4)


def _last():
    return native.lib().nvfp4_last_error().decode()


def test_quantize_validation():
    L = native.lib()
    q = lambda x=FAKE, dt=0, rows=4, cols=64, ld=64, br=1, codes=FAKE, sc=FAKE: \
        L.fp8_block_quantize(x, dt, rows, cols, ld, br, codes, sc, None)
    assert q(x=None) == 1 and "x is NULL" in _last()
    assert q(codes=None) == 1 and q(sc=None) == 1
    assert q(dt=2) == 1
    assert q(br=64) == 1 and "block_rows" in _last()
    assert q(rows=-1) == 1
    assert q(cols=48) == 2 and "multiple of 32" in _last()
    assert q(cols=0) == 2
    assert q(ld=32) == 1 and q(ld=68) == 1
    assert q(rows=1 << 28) == 2 and "2^27" in _last()
    assert q(x=MIS) == 3 and q(codes=MIS) == 3 and q(sc=MIS) == 3
    assert q(x=None, rows=0, codes=None, sc=None) == 0
    assert q(x=None, rows=0, cols=48, codes=None, sc=None) == 2


def test_linear_validation():
    L = native.lib()
    m = native.Fp8Matrix(FAKE.value, FAKE.value, 64, 96)
    ws = L.fp8_block_linear_workspace_size(40, 64, 96, 0)   # (up to 16 rows need none)
    assert ws > L.fp8_block_linear_workspace_size(40, 64, 96, 1)
    lin = lambda x=FAKE, xs=None, M=40, w=m, y=FAKE, dt=0, wsp=FAKE, wsb=ws: L.fp8_block_linear(
        x, xs, M, None if w is None else ctypes.byref(w), y, dt, wsp, wsb, None)
    assert lin(x=None) == 1 and lin(y=None) == 1 and lin(w=None) == 1
    assert lin(M=-1) == 1
    assert lin(M=(1 << 24) + 1) == 2
    assert lin(dt=5) == 1
    assert lin(w=native.Fp8Matrix(None, FAKE.value, 64, 96)) == 1 and "codes" in _last()
    assert lin(w=native.Fp8Matrix(FAKE.value, None, 64, 96)) == 1 and "scales" in _last()
    assert lin(w=native.Fp8Matrix(FAKE.value, FAKE.value, 0, 96)) == 1
    assert lin(w=native.Fp8Matrix(FAKE.value, FAKE.value, 64, 80)) == 2
    assert lin(w=native.Fp8Matrix(FAKE.value, FAKE.value, (1 << 24) + 1, 96)) == 2
    assert lin(w=native.Fp8Matrix(MIS.value, FAKE.value, 64, 96)) == 3
    assert lin(x=MIS) == 3 and lin(xs=MIS) == 3 and lin(y=MIS) == 3
    assert lin(wsb=ws - 256) == 4
    assert lin(wsp=None) == 1
    assert lin(x=None, y=None, M=0, wsp=None, wsb=0) == 0
    assert lin(x=None, y=None, M=0, wsp=None, wsb=0,
               w=native.Fp8Matrix(FAKE.value, FAKE.value, 64, 80)) == 2


def test_mlp_validation():
    L = native.lib()
    g = native.Fp8Matrix(FAKE.value, FAKE.value, 64, 96)
    d = native.Fp8Matrix(FAKE.value, FAKE.value, 96, 64)
    ws = L.fp8_block_mlp_workspace_size(4, 96, 64)
    assert ws > 0
    mlp = lambda x=FAKE, T=4, gate=g, up=g, down=d, y=FAKE, dt=0, wsb=ws: L.fp8_block_mlp(
        x, T, *(ctypes.byref(w) for w in (gate, up, down)), y, dt, FAKE, wsb, None)
    assert mlp(x=None) == 1 and mlp(y=None) == 1 and mlp(T=-1) == 1 and mlp(dt=2) == 1
    assert mlp(up=d) == 1 and "w_up" in _last()
    assert mlp(down=g) == 1
    assert mlp(gate=native.Fp8Matrix(FAKE.value, FAKE.value, 48, 96),
               up=native.Fp8Matrix(FAKE.value, FAKE.value, 48, 96),
               down=native.Fp8Matrix(FAKE.value, FAKE.value, 96, 48)) == 2   # I % 32
    assert mlp(T=(1 << 24) + 1) == 2
    assert mlp(x=MIS) == 3 and mlp(y=MIS) == 3
    assert mlp(wsb=ws - 256) == 4
    assert mlp(x=None, y=None, T=0, wsb=0) == 0


def test_workspace_sizes_of_empty_problems():
    L = native.lib()
    assert L.fp8_block_linear_workspace_size(0, 64, 96, 0) == 0
    assert L.fp8_block_mlp_workspace_size(0, 96, 64) == 0


def test_binding_refusals():
    """The binding's own checks, on host tensors (nothing reaches the library)."""
    x = torch.zeros((4, 96), dtype=torch.bfloat16)
    w, ws = torch.zeros((64, 96), dtype=torch.uint8), torch.ones((1, 1))
    with pytest.raises(ValueError, match="cuda"):
        native.fp8_block_quantize(x)
    with pytest.raises(ValueError, match="block_rows"):
        native.fp8_block_quantize(x, 64)
    with pytest.raises(ValueError, match="unit column stride"):
        native.fp8_block_quantize(x.t())
    with pytest.raises(ValueError, match=r"\[rows, cols\]"):
        native.fp8_block_quantize(x[0])
    with pytest.raises(ValueError, match="cuda"):
        native.fp8_block_linear(x, w, ws)
    with pytest.raises(ValueError, match="does not match"):
        native.fp8_block_linear(x[:, :64], w, ws)
    with pytest.raises(ValueError, match="scales"):
        native.fp8_block_linear(x, w, ws.repeat(2, 1))
    with pytest.raises(TypeError, match="bfloat16"):
        native.fp8_block_linear(x.float(), w, ws)
    with pytest.raises(TypeError, match="uint8"):
        native.fp8_block_linear(x, w, ws, x_scales=torch.ones((4, 1)))
    with pytest.raises(ValueError, match="x_scales"):
        native.fp8_block_linear(torch.zeros((4, 96), dtype=torch.uint8), w, ws,
                                x_scales=torch.ones((4, 2)))
    with pytest.raises(TypeError, match="uint8"):
        native.fp8_block_mlp(x, (w.int(), ws), (w, ws), (w, ws))


def test_sizes_past_the_kernels_ranges():
    """Offsets of sixteen rows, and scales of a batch, past what the kernels
    index: refused before anything else is looked at."""
    L = native.lib()
    big = 1 << 50
    lin = lambda M, N, K: L.fp8_block_linear(
        FAKE, None, M, ctypes.byref(native.Fp8Matrix(FAKE.value, FAKE.value, N, K)), FAKE, 0, FAKE,
        big, None)
    assert lin(1, 1, (1 << 27) + 32) == 2 and "2^27" in _last()
    assert lin(1 << 20, 1, 128 * 129) == 2 and "2^27" in _last()
    m = lambda n, k: ctypes.byref(native.Fp8Matrix(FAKE.value, FAKE.value, n, k))
    assert L.fp8_block_mlp(FAKE, 1 << 20, m(32, 128 * 129), m(32, 128 * 129), m(128 * 129, 32), FAKE, 0,
                           FAKE, big, None) == 2 and "2^27" in _last()
    assert L.fp8_block_mlp(FAKE, 1 << 20, m(128 * 129, 32), m(128 * 129, 32), m(32, 128 * 129), FAKE, 0,
                           FAKE, big, None) == 2 and "2^27" in _last()


def test_quantize_refuses_what_one_launch_cannot_hold():
    """f32 rows of 1 x 128 blocks go eight to a workgroup of 256: past 2^27 - 8
    of them a launch has 2^32 work-items or more."""
    L = native.lib()
    q = lambda dt, rows, br: L.fp8_block_quantize(FAKE, dt, rows, 128, 128, br, FAKE, FAKE, None)
    for rows in ((1 << 27) - 7, 1 << 27):
        assert q(native.DT_F32, rows, 1) == 2 and "2^27 - 8" in _last()
    assert q(native.DT_BF16, (1 << 27) + 1, 1) == 2 and "2^27" in _last()
    assert q(native.DT_F32, (1 << 27) + 1, 128) == 2 and "2^27" in _last()


MONOTONE = [(5120, 17408), (17408, 5120), (5120, 5120), (4096, 4096), (2048, 1056), (300, 2080),
            (17, 32), (32, 18464), (4112, 1024), (8192, 3936)]


@pytest.mark.parametrize("N,K", MONOTONE)
def test_workspace_of_a_batch_serves_smaller_ones(N, K):
    """A workspace allocated once, for the largest batch: also where fewer rows
    split K further, or change their form."""
    L = native.lib()
    rows = list(range(260)) + [*range(260, 2600, 13), 2048, 2049, 1 << 13, 1 << 16, 1 << 20, 1 << 24]
    rows.sort()
    for size in (lambda m: L.fp8_block_linear_workspace_size(m, N, K, 0),
                 lambda m: L.fp8_block_linear_workspace_size(m, N, K, 1),
                 lambda m: L.fp8_block_mlp_workspace_size(m, K, (N + 31) // 32 * 32)):
        sizes = [size(m) for m in rows]
        assert sizes == sorted(sizes)


def test_the_shapes_of_the_gpu_tests_take_the_tiles_they_name():
    """The plan is host code: a changed rule shows here, before the GPU tests of
    the larger tiles lose what they are for."""
    from test_gpu_fp8 import MLP_TILE_SHAPES, TILE_SHAPES
    for M, N, K, rows, parts in TILE_SHAPES:
        assert native.fp8_debug_plan(M, N, K) == (rows, parts), (M, N, K)
    for T, H, I, rows, parts in MLP_TILE_SHAPES:
        assert native.fp8_debug_plan(T, I, H, gate_up=True) == (rows, parts), (T, H, I)
    for shapes in (TILE_SHAPES, MLP_TILE_SHAPES):
        assert {(s[3], s[4] > 1) for s in shapes} == {(128, False), (128, True), (192, False),
                                                      (192, True)}
    assert native.fp8_debug_plan(64, 4096, 4096) == (0, 0)
    assert native.fp8_debug_plan(32, 4096, 4096, gate_up=True) == (0, 0)


def test_linear_refuses_an_output_over_its_input():
    """Where the product reads x itself, workgroups that are done would overwrite
    what others still quantise."""
    L = native.lib()
    m = native.Fp8Matrix(1 << 30, 1 << 29, 256, 256)
    lin = lambda x, y, xs=None, M=4, dt=0: L.fp8_block_linear(
        x, xs, M, ctypes.byref(m), y, dt, None, 0, None)
    row = 512                                                   # bytes of a bf16 row
    for y in (1 << 20, (1 << 20) + 3 * row, (1 << 20) - 3 * row):
        assert lin(1 << 20, y) == 1 and "overlap" in _last()
    for y in ((1 << 20) + 3 * 256, (1 << 20) - 7 * 512):        # codes in, f32 out
        assert lin(1 << 20, y, xs=1 << 25, dt=1) == 1 and "overlap" in _last()
