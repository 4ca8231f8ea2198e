"""GPU checks of the state space layer's values at the ends of its inputs' ranges: magnitudes that
differ within a row, far negative gates, rates and steps at the ends of fp32, empty calls and
unusual sequence tables."""
import ctypes

import pytest
import torch

import gated_deltanet_layer_02_b200 as gdn
from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


@pytest.mark.parametrize("N", [1, 3, 40])
@DTYPES
def test_sequences_without_a_token_need_no_rows(dtype, N):
    # the C call with num_tokens 0 may pass NULL for everything that belongs to tokens, the conv
    # weights among them: the states are handed on
    ensure_built()
    dims = gdn.SsmDims(4, 2, 64, 128)
    S0, conv0 = torch.randn(N, 4, 64, 128).cuda(), torch.randn(N, 3, dims.channels).to(dtype).cuda()
    SN, convN = torch.full_like(S0, 3.0), torch.full_like(conv0, 3.0)
    cu, a_log = torch.zeros(N + 1, dtype=torch.int32).cuda(), torch.zeros(4).cuda()
    ws = torch.empty(gdn.ssm_prefill_workspace_size(N, 0, dtype, dims), dtype=torch.uint8).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    rc = gdn.lib().gdn_ssm_prefill(
        ctypes.byref(dims), gdn.GDN_BF16 if dtype == BF else gdn.GDN_F32, None, None, None, None,
        None, a_log.data_ptr(), None, None, cu.data_ptr(), N, 0, S0.data_ptr(), SN.data_ptr(),
        conv0.data_ptr(), convN.data_ptr(), None, ws.data_ptr(), ws.numel(), status.data_ptr(),
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == gdn.GDN_OK and int(status.item()) == 0
    assert torch.equal(SN, S0) and torch.equal(convN, conv0)
