"""Refusals of the int8 operators and of the RMS norm: the documented status
before anything is enqueued (C ABI), and the binding's checks (no GPU needed)."""
import ctypes
import os

import pytest
import torch

from nvfp4_routed_expert_amd import native

pytestmark = pytest.mark.skipif(not os.path.exists(native.LIB_PATH),
                                reason="library not built")

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 4)
A, B, C, D, E, F = (i << 40 for i in range(1, 7))   # far apart, never dereferenced


def _last():
    return native.lib().nvfp4_last_error().decode()


def mat(n, k, codes=A, scales=B):
    return native.Int8Matrix(codes, scales, n, k)


def test_quantize_validation():
    L = native.lib()
    q = lambda x=A, dt=0, rows=4, cols=64, ld=64, codes=B, sc=C: \
        L.int8_quantize(x, dt, rows, cols, ld, codes, sc, None)
    assert q(x=None) == 1 and "x is NULL" in _last()
    assert q(codes=None) == 1 and q(sc=None) == 1
    assert q(dt=2) == 1 and q(dt=-1) == 1
    assert q(rows=-1) == 1
    assert q(rows=(1 << 24) + 1) == 2
    assert q(cols=48) == 2 and "multiple of 32" in _last()
    assert q(cols=0) == 2 and q(cols=(1 << 27) + 32, ld=1 << 28) == 2
    assert q(ld=32) == 1 and q(ld=68) == 1 and q(ld=(1 << 31) + 8) == 2
    assert q(x=A + 4) == 3 and q(codes=B + 8) == 3 and q(sc=C + 4) == 3
    # codes or scales over x, scales over codes, in the first and the last bytes
    last = A + (3 * 96 + 64) * 2 - 16
    assert q(codes=A) == 1 and "overlap" in _last()
    assert q(ld=96, codes=last) == 1 and q(ld=96, sc=last) == 1
    assert q(codes=A - 3 * 64) == 1 and q(sc=B + 240) == 1
    assert q(x=None, rows=0, codes=None, sc=None) == 0
    assert q(x=None, rows=0, cols=48, codes=None, sc=None) == 2


def test_linear_validation():
    L = native.lib()
    size = L.int8_linear_workspace_size
    need = size(40, 64, 96, 0)
    assert need > size(40, 64, 96, 1)
    lin = lambda x=C, xs=None, M=40, w=mat(64, 96), y=D, dt=0, wsp=E, wsb=1 << 30: L.int8_linear(
        x, xs, M, None if w is None else ctypes.byref(w), y, dt, wsp, wsb, None)
    assert lin(x=None) == 1 and lin(y=None) == 1 and lin(w=None) == 1
    assert lin(M=-1) == 1 and lin(M=(1 << 24) + 1) == 2
    assert lin(dt=5) == 1
    assert lin(w=mat(64, 96, codes=None)) == 1 and "codes" in _last()
    assert lin(w=mat(64, 96, scales=None)) == 1 and "scales" in _last()
    assert lin(w=mat(0, 96)) == 1 and lin(w=mat((1 << 24) + 1, 96)) == 2
    assert lin(w=mat(64, 80)) == 2 and lin(w=mat(64, 0)) == 2
    assert lin(w=mat(64, 131072)) == 2 and "131040" in _last()
    assert lin(w=mat(64, 96, codes=A + 8)) == 3 and lin(w=mat(64, 96, scales=B + 8)) == 3
    assert lin(M=1 << 24, w=mat(4097, 32)) == 2 and "2^36" in _last()
    assert lin(x=C + 4) == 3 and lin(xs=E + 4) == 3 and lin(y=D + 4) == 3
    assert lin(wsb=need - 256) == 4 and lin(wsp=None) == 1 and lin(wsp=E + 8) == 3
    row = 96 * 2
    for y in (C, C + 39 * row, C - 39 * 128):                        # bf16 in, bf16 out
        assert lin(y=y) == 1 and "overlaps x" in _last()
    for y in (C + 39 * 96, C - 39 * 256):                            # codes in, f32 out
        assert lin(y=y, xs=E, dt=1) == 1 and "overlaps x" in _last()
    assert lin(y=F, xs=F + 16) == 1 and "x_scales" in _last()
    assert lin(y=E + 64) == 1 and "workspace" in _last()
    assert lin(y=A + 64) == 1 and "w->codes" in _last()
    assert lin(y=B + 64) == 1 and "w->scales" in _last()
    for at, name in ((C, "x"), (A, "w->codes"), (B, "w->scales")):
        assert lin(wsp=at) == 1 and "workspace overlaps " + name in _last()
    assert lin(x=None, y=None, M=0, wsp=None, wsb=0) == 0
    assert lin(x=None, y=None, M=0, wsp=None, wsb=0, w=mat(64, 80)) == 2


def test_mlp_validation():
    L = native.lib()
    g, d = mat(64, 96), mat(96, 64)
    need = L.int8_mlp_workspace_size(4, 96, 64, 0)
    # (few rows are quantised inside the product)
    assert L.int8_mlp_workspace_size(100, 96, 64, 0) > L.int8_mlp_workspace_size(100, 96, 64, 1) > 0
    mlp = lambda x=C, xs=None, T=4, gate=g, up=g, down=d, y=D, dt=0, wsb=1 << 30: L.int8_mlp(
        x, xs, T, *(ctypes.byref(w) for w in (gate, up, down)), y, dt, E, wsb, None)
    assert mlp(x=None) == 1 and mlp(y=None) == 1 and mlp(T=-1) == 1 and mlp(dt=2) == 1
    assert mlp(up=d) == 1 and "w_up" in _last()
    assert mlp(down=g) == 1
    assert mlp(gate=mat(48, 96), up=mat(48, 96), down=mat(96, 48)) == 2     # I % 32
    assert mlp(T=(1 << 24) + 1) == 2
    big = mat(4128, 32)
    assert mlp(T=1 << 24, gate=big, up=big, down=mat(32, 4128)) == 2 and "2^36" in _last()
    assert mlp(x=C + 4) == 3 and mlp(y=D + 4) == 3 and mlp(xs=F + 4) == 3
    assert mlp(wsb=need - 256) == 4
    assert mlp(y=C + 16) == 1 and mlp(xs=D, y=D) == 1 and mlp(y=E) == 1
    for name in ("w_gate", "w_up", "w_down"):
        m = mat(96, 64, F, F + (1 << 30)) if name == "w_down" else mat(64, 96, F, F + (1 << 30))
        for y in (F + 16, F + (1 << 30)):
            assert mlp(**{name[2:]: m}, y=y) == 1 and name in _last()
    assert mlp(x=None, y=None, T=0, wsb=0) == 0


def norm_args(**kw):
    a = native.RmsNormArgs(x=A, x_dtype=0, ld_x=64, residual=B, residual_dtype=0, ld_residual=64,
                           residual_out=C, ld_residual_out=64, weight=D, weight_dtype=0, eps=1e-6,
                           y=E, y_dtype=0, format=2, codes=F, scales=F + (1 << 30))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def norm(T=4, H=64, **kw):
    return native.lib().rms_norm_quantize(ctypes.byref(norm_args(**kw)), T, H, None)


def test_norm_validation():
    assert native.lib().rms_norm_quantize(None, 4, 64, None) == 1
    assert norm(x=None) == 1 and norm(weight=None) == 1
    assert norm(y=None, format=0, codes=None, scales=None) == 1 and "no codes" in _last()
    assert norm(format=3) == 1 and norm(format=-1) == 1
    assert norm(codes=None) == 1 and norm(scales=None) == 1
    assert norm(format=0) == 1 and norm(format=0, codes=None) == 1       # codes nobody asked for
    assert norm(residual=None) == 1 and norm(residual_out=None) == 1
    for name in ("x_dtype", "residual_dtype", "weight_dtype", "y_dtype"):
        assert norm(**{name: 2}) == 1
    assert norm(T=-1) == 1 and norm(T=(1 << 24) + 1) == 2
    assert norm(H=48) == 2 and norm(H=0) == 2
    assert norm(H=(1 << 27) + 32, ld_x=1 << 28, ld_residual=1 << 28, ld_residual_out=1 << 28) == 2
    for name in ("ld_x", "ld_residual", "ld_residual_out"):
        assert norm(**{name: 32}) == 1 and norm(**{name: 68}) == 1
        assert norm(**{name: (1 << 31) + 8}) == 2
    for eps in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -127, 2.0 ** 126):
        assert norm(eps=eps) == 1 and "eps" in _last()
    for name in ("x", "residual", "residual_out", "weight", "y", "codes", "scales"):
        assert norm(**{name: getattr(norm_args(), name) + 8}) == 3 and name in _last()
    assert norm(T=0) == 0 and norm(T=0, x=None, y=None, codes=None, scales=None, residual=None,
                                   residual_out=None) == 0
    assert norm(T=0, H=48) == 2


def test_norm_refuses_overlaps():
    """No output over an input or another output, but for the residual replaced
    by the sum, or x by it, in the same layout."""
    for out in ("residual_out", "y", "codes", "scales"):
        for other in ("x", "residual", "weight", "y", "codes", "scales", "residual_out"):
            if out == other:
                continue
            at = getattr(norm_args(), other)
            exact = out == "residual_out" and other in ("x", "residual")
            if not exact:
                assert norm(**{out: at}) == 1 and "overlaps" in _last(), (out, other)
            # (eight rows: 32 bytes of scales)
            assert norm(T=8, **{out: at + 16}) == 1 and "overlaps" in _last(), (out, other)
    # the same place in another layout
    assert norm(residual_out=B, ld_residual_out=72) == 1
    assert norm(residual_out=A, residual_dtype=1) == 1
    assert norm(residual_out=A, ld_x=72) == 1
    # the last element of a strided x
    assert norm(ld_x=96, codes=A + (3 * 96 + 64) * 2 - 16) == 1


def test_workspace_sizes():
    L = native.lib()
    assert L.int8_linear_workspace_size(0, 64, 96, 0) == 0
    assert L.int8_mlp_workspace_size(0, 96, 64, 0) == 0
    assert L.int8_linear_workspace_size(1 << 25, 64, 96, 0) == 0      # refused sizes
    assert L.int8_mlp_workspace_size(4, 131072, 64, 0) == 0


MONOTONE = [(5120, 17408), (17408, 5120), (5120, 5120), (4096, 4096), (2048, 1056), (300, 2080),
            (17, 32), (32, 18464), (4112, 1024), (8192, 3936), (64, 131040)]


@pytest.mark.parametrize("N,K", MONOTONE)
def test_workspace_of_a_batch_serves_smaller_ones(N, K):
    L = native.lib()
    rows = list(range(260)) + [*range(260, 2600, 13), 2048, 2049, 1 << 13, 1 << 16, 1 << 20, 1 << 22]
    rows.sort()
    for size in (lambda m: L.int8_linear_workspace_size(m, N, K, 0),
                 lambda m: L.int8_linear_workspace_size(m, N, K, 1),
                 lambda m: L.int8_mlp_workspace_size(m, K, (N + 31) // 32 * 32, 0),
                 lambda m: L.int8_mlp_workspace_size(m, K, (N + 31) // 32 * 32, 1)):
        sizes = [size(m) for m in rows]
        assert sizes == sorted(sizes)


def test_binding_refusals():
    """The binding's own checks, on host tensors (nothing reaches the library)."""
    x = torch.zeros((4, 96), dtype=torch.bfloat16)
    w, ws = torch.zeros((64, 96), dtype=torch.int8), torch.ones(64)
    with pytest.raises(ValueError, match="cuda"):
        native.int8_quantize(x)
    with pytest.raises(ValueError, match="unit column stride"):
        native.int8_quantize(x.t())
    with pytest.raises(ValueError, match=r"\[rows, cols\]"):
        native.int8_quantize(x[0])
    with pytest.raises(ValueError, match="cuda"):
        native.int8_linear(x, w, ws)
    with pytest.raises(ValueError, match="does not match"):
        native.int8_linear(x[:, :64], w, ws)
    with pytest.raises(ValueError, match="scales"):
        native.int8_linear(x, w, ws[:32])
    with pytest.raises(TypeError, match="int8"):
        native.int8_linear(x, w.view(torch.uint8), ws)
    with pytest.raises(TypeError, match="bfloat16"):
        native.int8_linear(x.float(), w, ws)
    with pytest.raises(TypeError, match="int8"):
        native.int8_linear(x, w, ws, x_scales=torch.ones(4))
    with pytest.raises(ValueError, match="x_scales"):
        native.int8_linear(x.to(torch.int8), w, ws, x_scales=torch.ones(3))
    with pytest.raises(TypeError, match="int8"):
        native.int8_mlp(x, (w.int(), ws), (w, ws), (w, ws))
    with pytest.raises(ValueError, match="does not match"):
        native.int8_mlp(x[:, :32], (w, ws), (w, ws), (w, ws))
    g = torch.ones(96)
    with pytest.raises(ValueError, match="codes must be"):
        native.rms_norm_quantize(x, g, codes="int4")
    with pytest.raises(ValueError, match="nothing to compute"):
        native.rms_norm_quantize(x, g)
    with pytest.raises(ValueError, match="cuda"):
        native.rms_norm_quantize(x, g, codes="int8")
    with pytest.raises(ValueError, match=r"\[T, H\]"):
        native.rms_norm_quantize(x[0], g, codes="int8")


def test_norm_refuses_outputs_nobody_asked_for():
    x, g = torch.zeros((4, 96), dtype=torch.bfloat16), torch.ones(96)
    class Cuda(torch.Tensor):          # a host tensor that passes for one on a device
        is_cuda = True
    x, g = x.as_subclass(Cuda), g.as_subclass(Cuda)
    o = lambda **k: native.RmsNorm(*(k.get(n) for n in ("y", "codes", "scales", "residual")))
    for kw, out in (({"codes": "int8"}, o(y=x)), ({"codes": "int8"}, o(residual=x)),
                    ({"y_dtype": torch.float32}, o(codes=x)), ({"y_dtype": torch.float32}, o(scales=x))):
        with pytest.raises(ValueError, match="not asked for"):
            native.rms_norm_quantize(x, g, out=out, **kw)


def test_the_shapes_of_the_gpu_tests_take_the_tiles_they_name():
    """The plan is host code: a changed rule shows here, before the GPU tests of
    the tiles lose what they are for."""
    from test_gpu_int8 import MLP_TILE_SHAPES, MLP_TWO_LAUNCHES, TILE_SHAPES, TWO_LAUNCHES
    for shapes, gate_up in ((TWO_LAUNCHES, False), (MLP_TWO_LAUNCHES, True)):
        for M, N, K, rows, columns, main in shapes:
            assert main < N
            assert native.int8_debug_plan(M, N, K, gate_up) == (rows, columns, 1, main)
    for M, N, K, *plan in TILE_SHAPES:
        assert native.int8_debug_plan(M, N, K) == (*plan, N), (M, N, K)
    for T, I, H, *plan in MLP_TILE_SHAPES:
        assert native.int8_debug_plan(T, I, H, gate_up=True) == (*plan, I), (T, I, H)
    tiles = {(64, 64), (64, 128), (64, 256), (128, 128), (128, 256), (192, 64), (192, 128),
             (192, 256), (256, 256)}
    kinds = lambda shapes: {(s[3], s[4], s[5] > 1) for s in shapes}
    assert kinds(TILE_SHAPES) == {(*t, split) for t in tiles for split in (False, True)}
    assert kinds(MLP_TILE_SHAPES) == {(*t, split) for t in tiles if t[1] > 64
                                      for split in (False, True)}
    assert native.int8_debug_plan(16, 4096, 4096) == (0, 0, 0, 0)
    assert native.int8_debug_plan(32, 4096, 4096, gate_up=True) == (0, 0, 0, 0)
    for bad in ((0, 64, 64), (64, 0, 64), (64, 64, 0), (-1, 64, 64), (2 ** 24 + 1, 64, 64),
                (64, 2 ** 24 + 1, 64), (64, 64, 131072), (2 ** 19, 2 ** 18, 64),
                (2 ** 62, 2 ** 62, 2 ** 62)):
        assert native.int8_debug_plan(*bad) == (0, 0, 0, 0)
    assert native.lib().int8_debug_plan(0, 64, 64, 64, None, None, None) > 0


@pytest.mark.parametrize("N,K", MONOTONE)
def test_parts_fit_the_workspace(N, K):
    """The sums of a call's parts fit what the query of any larger batch names
    for them (what is left of the workspace holds x's codes and scales)."""
    L = native.lib()
    for gate_up in (False, True):
        n = (N + 31) // 32 * 32 if gate_up else N
        for M in [*range(1, 700, 3), 1023, 1500, 2049, 5000]:
            parts = native.int8_debug_plan(M, n, K, gate_up)[2]
            if parts < 2:
                continue
            words = parts * M * n * (2 if gate_up else 1)
            size = L.int8_mlp_workspace_size(M, K, n, 1) if gate_up else \
                L.int8_linear_workspace_size(M, n, K, 1)
            assert size >= 4 * words, (M, n, K, gate_up)
