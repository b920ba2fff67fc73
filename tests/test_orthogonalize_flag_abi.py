"""The testing flag of the orthogonalisation's iterations changes no check of them."""
import ctypes

import pytest

import sparse_mixture_experts_topk_gb300 as moe

A = 1 << 20          # an aligned address that is never read
STALL = moe.MOE_ORTHOGONALIZE_TEST_WAIT_TIMEOUT


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_mixture_experts_topk_gb300 import build
    build.build()


@pytest.mark.parametrize("iterations", [STALL, 17 | STALL, -1, 5 | 2 * (STALL >> 2), -2 ** 31 | STALL | 5])
def test_iterations_are_checked_without_the_flag(iterations):
    L = moe.lib()
    f32 = moe.MOE_F32
    assert L.moe_orthogonalize(A, f32, 2, 30, 40, iterations, A, f32, A, 1 << 30, None) == moe.MOE_ERR_INVALID
    t = (moe.MoeMuonTensor * 1)(moe.MoeMuonTensor(A, A, A, A, 2, 30, 40, 0.1, 1.0))
    h = moe.MoeMuonParams(0.1, 0.9, 1, iterations)
    assert L.moe_muon_step(t, 1, f32, ctypes.byref(h), None, None, A, 1 << 30, None) == moe.MOE_ERR_INVALID


def test_a_flagged_call_is_checked_as_any_other():
    L = moe.lib()
    assert L.moe_orthogonalize(A, moe.MOE_F32, 2, 30, 40, 5 | STALL, A, moe.MOE_F32, None, 0, None) == moe.MOE_ERR_WORKSPACE
    t = (moe.MoeMuonTensor * 1)(moe.MoeMuonTensor(A, A, A, A, 2, 30, 40, 0.1, 1.0))
    h = moe.make_muon(0.1, iterations=5 | STALL)
    assert L.moe_muon_step(t, 1, moe.MOE_F32, ctypes.byref(h), None, None, None, 0, None) == moe.MOE_ERR_WORKSPACE
