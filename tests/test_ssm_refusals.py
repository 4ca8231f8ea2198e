"""Refusals of the state space calls that need no GPU (addresses that are never read)."""
import ctypes

import pytest

import gated_deltanet_layer_02_b200 as gdn
from gated_deltanet_layer_02_b200 import build as gdn_build

A, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)
DIMS = ctypes.byref(gdn.SsmDims())


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


@pytest.mark.parametrize("dtype", [gdn.GDN_F32, gdn.GDN_BF16])
@pytest.mark.parametrize("which", ["cu_seqlens", "slot_idx", "dev_status"])
def test_index_arrays_are_aligned_to_their_type(L, which, dtype):
    cu, slot, status = (ODD if which == k else A for k in ("cu_seqlens", "slot_idx", "dev_status"))
    if which != "slot_idx":
        assert L.gdn_ssm_prefill(DIMS, dtype, A, A, None, A, None, A, None, None, cu, 1, 16, None,
                                 None, None, None, A, A, 1 << 40, status, None) == \
            gdn.GDN_ERR_INVALID_ARG
    assert L.gdn_ssm_prefill_slots(DIMS, dtype, A, A, None, A, None, A, None, None, cu, 1, 16, slot,
                                   4, A, A, A, A, 1 << 40, status, None) == gdn.GDN_ERR_INVALID_ARG
    if which != "cu_seqlens":
        assert L.gdn_ssm_decode_step(DIMS, dtype, 0, A, A, None, A, None, A, None, None, A, A, slot,
                                     4, 2, A, status, None) == gdn.GDN_ERR_INVALID_ARG


def test_debug_faults_of_the_prefill_are_known(L):
    for fault, want in ((gdn.GDN_FAULT_SKIP_SSM_PRODUCT, gdn.GDN_OK),
                        (gdn.GDN_FAULT_SKIP_SSM_SEG_LOAD, gdn.GDN_OK),
                        (gdn.GDN_FAULT_SKIP_SSM_LOAD, gdn.GDN_OK),
                        (gdn.GDN_FAULT_SKIP_SSM_LOAD + 1, gdn.GDN_ERR_INVALID_ARG),
                        (-1, gdn.GDN_ERR_INVALID_ARG)):
        opts = gdn.DebugOptions(5000, 0, 0, fault, 0)
        assert L.gdn_debug_set(ctypes.byref(opts)) == want
        assert L.gdn_debug_set(None) == gdn.GDN_OK
