"""Operands and results that are slices of one wider matrix: which addresses share memory (no GPU; where
nothing is refused the calls end at the missing device)."""
import pytest

import blackwell_tensor_core_02_gb300 as g
from blackwell_tensor_core_02_gb300 import grouped

torch = pytest.importorskip("torch")

INVALID = -1
P = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    import ctypes

    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    lib = ctypes.CDLL(grouped.load_grouped()._name)
    lib.norm_checkpoint_forward.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, i64, i64, f32, i32, i32, vp]
    lib.norm_checkpoint_restore.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
    lib.norm_checkpoint_backward.argtypes = [vp, i64, vp, vp, vp, vp, vp, i64, vp, vp, i64, i64, i32, i32, vp, i64, vp]
    return lib


# 4 rows of 64 halves, 256 bytes apart: where another slice of such rows may begin
PLACES = [(128, False), (126, True), (2, True), (130, True), (-128, False), (-126, True), (3 * 256 + 128, False),
          (2 * 256, True), (4 * 256, False), (-3 * 256 - 128, False)]


@pytest.mark.parametrize("off,refused", PLACES)
def test_checkpoints(lib, off, refused):
    keep = lib.norm_checkpoint_forward(P, 128, None, None, P + off, 128, 3 * P, 4 * P, 5 * P, 4, 64, 1e-5, 0, 0, None)
    assert (keep == INVALID) == refused
    grad = lib.norm_checkpoint_backward(P, 128, 2 * P, 3 * P, None, 4 * P, P + off, 128, 6 * P, 7 * P, 4, 64, 0, 0, 8 * P, 1 << 20, None)
    assert (grad == INVALID) == refused


def test_checkpoints_of_other_strides(lib):
    def keep(y, xs=128, ys=128, rows=4, codes=3 * P):
        return lib.norm_checkpoint_forward(P, xs, None, None, y, ys, codes, 4 * P, 5 * P, rows, 64, 1e-5, 0, 0, None)

    assert keep(P + 128, ys=136) == keep(P - 128, xs=0) == keep(P + 128, xs=64, ys=64) == keep(P + 64, rows=1) == INVALID
    assert keep(P + 128, codes=P + 128) == keep(P + 128, codes=P) == INVALID
    # what a restored row shares with the codes is refused wherever it lies
    assert lib.norm_checkpoint_restore(P, 2 * P, None, None, P + 128, 128, 4, 64, 0, 0, None) == INVALID


@pytest.mark.parametrize("off,refused", [(64, False), (80, False), (48, True), (16, True), (0, True), (96, True), (-80, False), (-64, True),
                                         (3 * 160 + 64, False), (4 * 160, False), (160 + 80, False)])
def test_rows_of_other_widths(lib, off, refused):
    """A's rows of 32 halves and D's of 40, 80 halves (160 bytes) apart."""
    nt = lambda a, d: grouped.load_grouped().grouped_gemm_nt(a, 80, 2 * P, 32, 40 * 32, 3 * P, 0, d, 80, 4, 3, 40, 32, 0, 1, None, None)
    nn = lambda a, d: grouped.load_grouped().grouped_gemm_nn(d, 80, 2 * P, 32, 40 * 32, 3 * P, 0, a, 80, 4, 3, 40, 32, 0, 1, None, None)
    lora = lambda x, d: grouped.load_grouped().gemm_lora_nt(x, 80, 2 * P, 32, 4 * P, 32, 8 * 32, 5 * P, 8, 40 * 8, None, 3 * P, 0, 6 * P, d, 80,
                                                            4, 3, 2, 40, 32, 8, 0, 7 * P, 1 << 16, None, None)
    for call in (nt, nn, lora):
        assert (call(P, P + off) == INVALID) == refused
