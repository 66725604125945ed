"""CPU checks of the MoE operators' calls at the edges of their contracts: what they accept and refuse
before anything is launched."""
import ctypes

import pytest

import moe_grouped_gemm_02_gb300 as dg
from moe_grouped_gemm_02_gb300 import build as dg_build

GOOD = ctypes.c_void_p(0x10000)         # never dereferenced: every case returns before a launch
INVALID, OK = 1, 0


@pytest.fixture(scope="module")
def lib():
    dg_build.build()
    return dg.load_library()


def test_epilogue_calls_without_rows_take_null(lib):
    # tensors without elements have a null pointer; the weights, which have some, may not
    for b, sfb, want in ((GOOD, GOOD, OK), (None, GOOD, INVALID), (GOOD, None, INVALID)):
        assert lib.dg_fp8_gemm_nt_act(None, None, b, sfb, GOOD, None, None, None, 0, 512, 256, 4, 1, None) == want
        assert lib.dg_m_grouped_fp8_gemm_nt_contiguous_act(None, None, b, sfb, GOOD, None, None, None, None, 0, 512, 256, 4, 4, 1,
                                                           None) == want
        assert lib.dg_m_grouped_fp8_gemm_nt_masked_act(None, None, b, sfb, GOOD, None, None, None, GOOD, 4, 0, 512, 256, 4, 1,
                                                       None) == want
    assert lib.dg_m_grouped_fp8_gemm_nt_masked_act(None, None, GOOD, GOOD, None, None, None, None, None, 4, 0, 512, 256, 0, 0,
                                                   None) == INVALID      # masked_m has an entry per group
    # with rows every one of them is needed
    for hole in range(4):
        a, sfa, d, m = (None if i == hole else GOOD for i in range(4))
        assert lib.dg_m_grouped_fp8_gemm_nt_contiguous_act(a, sfa, GOOD, GOOD, None, None, None, d, m, 128, 512, 256, 4, 0, 0,
                                                           None) == INVALID


def test_activation_gradient_without_rows_takes_null(lib):
    for G in (1, 5):
        assert lib.dg_act_backward(None, None, None, None, None, None, 0, 256, G, 4, None) == OK
    assert lib.dg_act_backward(GOOD, GOOD, None, GOOD, None, None, 128, 256, 5, 4, None) == INVALID
