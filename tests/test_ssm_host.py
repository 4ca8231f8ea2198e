"""Refusals of the state space and table calls that need no GPU: the C ABI with addresses that
are never read, and the binding with CPU tensors."""
import ctypes

import pytest
import torch

import gated_deltanet_layer_02_b200 as gdn
from gated_deltanet_layer_02_b200 import build as gdn_build

P = ctypes.c_void_p
A, MIS = P(1 << 20), P((1 << 20) + 8)
BAD, UNSUP, WS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


def ref(**kw):
    return ctypes.byref(gdn.SsmDims(**kw))


def test_shapes(L):
    assert gdn.ssm_conv_channels(gdn.SsmDims(64, 8, 64, 128)) == 64 * 64 + 2 * 8 * 128
    assert gdn.SsmDims(24, 2, 64, 64).channels == 24 * 64 + 2 * 2 * 64
    assert L.gdn_ssm_conv_channels(None) == -1
    f = L.gdn_ssm_prefill_workspace_size
    assert 0 < f(ref(), 1, 1, 100) < f(ref(), 1, 1, 1000)
    assert f(ref(), 1, 0, 0) > 0 and f(ref(), 0, 0, 0) > 0
    assert f(None, 1, 1, 100) == 0 and f(ref(), 1, -1, 5) == 0 and f(ref(), 4, 1, 5) == 0
    assert f(ref(head_dim=96), 1, 1, 100) == 0


def prefill(L, dims, dtype=1, x=A, w=A, b=None, dt=A, a_log=A, z=None, cu=A, N=1, T=16, S0=None,
            out=A, ws=A, ws_bytes=1 << 40):
    return L.gdn_ssm_prefill(dims, dtype, x, w, b, dt, None, a_log, None, z, cu, N, T, S0, None,
                             None, None, out, ws, ws_bytes, None, None)


def test_prefill_refusals(L):
    d = ref()
    assert prefill(L, None) == BAD
    for kw, want in ((dict(num_heads=0), BAD), (dict(num_heads=9, num_groups=2), BAD),
                     (dict(num_groups=-1), BAD), (dict(head_dim=96), UNSUP),
                     (dict(head_dim=32), UNSUP), (dict(state_dim=256), UNSUP),
                     (dict(state_dim=16), UNSUP), (dict(conv_kernel=3), UNSUP),
                     (dict(dt_min=-1.0), BAD), (dict(dt_min=2.0, dt_max=1.0), BAD),
                     (dict(dt_min=float("nan")), BAD), (dict(dt_max=float("nan")), BAD),
                     (dict(num_heads=1 << 20), UNSUP)):
        assert prefill(L, ref(**kw)) == want, kw
    for kw, want in ((dict(dtype=2), UNSUP), (dict(x=None), BAD), (dict(w=None), BAD),
                     (dict(dt=None), BAD), (dict(a_log=None), BAD), (dict(cu=None), BAD),
                     (dict(out=None), BAD), (dict(x=MIS), BAD), (dict(b=MIS), BAD),
                     (dict(z=MIS), BAD), (dict(S0=MIS), BAD), (dict(N=-1), BAD), (dict(T=-1), BAD),
                     (dict(N=0), BAD), (dict(ws=None), WS), (dict(ws_bytes=64), WS),
                     (dict(ws=P((1 << 20) + 16)), BAD), (dict(N=1 << 30), UNSUP)):
        assert prefill(L, d, **kw) == want, kw
    assert prefill(L, d, N=0, T=0, x=None, w=None, dt=None, a_log=None, cu=None,
                   out=None) == gdn.GDN_OK


def test_slots_refusals(L):
    def call(S=A, slot=A, slots=4, N=2, conv=A):
        return L.gdn_ssm_prefill_slots(ref(), 1, A, A, None, A, None, A, None, None, A, N, 16, slot,
                                       slots, S, conv, A, A, 1 << 40, None, None)
    assert call(S=None) == BAD
    assert call(S=MIS) == BAD
    assert call(conv=MIS) == BAD
    assert call(slots=-1) == BAD
    assert call(slot=None, slots=1) == BAD


def test_decode_refusals(L):
    def call(dims=ref(), dtype=1, state=0, x=A, w=A, dt=A, a_log=A, conv=A, S=A, slot=A, slots=4,
             B=2, out=A):
        return L.gdn_ssm_decode_step(dims, dtype, state, x, w, None, dt, None, a_log, None, None,
                                     conv, S, slot, slots, B, out, None, None)
    for kw, want in ((dict(dims=None), BAD), (dict(dtype=3), UNSUP), (dict(state=3), UNSUP),
                     (dict(x=None), BAD), (dict(w=None), BAD), (dict(dt=None), BAD),
                     (dict(a_log=None), BAD), (dict(conv=None), BAD), (dict(S=None), BAD),
                     (dict(out=None), BAD), (dict(S=MIS), BAD), (dict(conv=MIS), BAD),
                     (dict(B=-1), BAD), (dict(slots=-1), BAD), (dict(slot=None, slots=1), BAD),
                     (dict(B=1 << 30), UNSUP), (dict(dims=ref(num_heads=2048, num_groups=1)), UNSUP)):
        assert call(**kw) == want, kw
    assert call(B=0, x=None, w=None, dt=None, a_log=None, conv=None, S=None, out=None) == gdn.GDN_OK


def test_tables_refusals(L):
    H = P(1 << 21)

    def call(ctx=A, new=A, slot=A, slots=4, N=2, table=A, width=8, free=A, nfree=5, head=A, page=64,
             rows=10, cu=A, pos=A, mp=A, head_out=H, status=None):
        return L.gdn_batch_tables(ctx, new, slot, slots, N, table, width, free, nfree, head, page,
                                  rows, cu, pos, mp, head_out, status, None)
    for kw in (dict(N=-1), dict(slots=-1), dict(width=-1), dict(nfree=-1), dict(rows=-1),
               dict(page=0), dict(page=-16), dict(cu=None), dict(head=None), dict(head_out=None),
               dict(head_out=A), dict(new=None), dict(table=None), dict(free=None),
               dict(slot=None, slots=1), dict(mp=P((1 << 20) + 4)), dict(new=P((1 << 20) + 2))):
        assert call(**kw) == BAD, kw


def test_status_string():
    assert gdn.status_string(gdn.GDN_ERR_PAGES) == "not enough free pages"


def test_binding_refusals(L):
    d = gdn.SsmDims(2, 1)
    T, Cc, bf = 6, d.channels, torch.bfloat16
    x, dt, a_log = torch.zeros(T, Cc, dtype=bf), torch.zeros(T, 2), torch.zeros(2)
    w, cu = torch.zeros(Cc, 4, dtype=bf), torch.tensor([0, T], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.ssm_prefill(x, dt, a_log, cu, w, dims=d)
    with pytest.raises(ValueError, match="x holds"):
        gdn.ssm_prefill(x[:, :64], dt, a_log, cu, w, dims=d)
    with pytest.raises(ValueError, match="dt holds"):
        gdn.ssm_prefill(x, dt[:3], a_log, cu, w, dims=d)
    with pytest.raises(ValueError, match="conv_w holds"):
        gdn.ssm_prefill(x, dt, a_log, cu, w[:, :3], dims=d)
    with pytest.raises(ValueError, match="z holds"):
        gdn.ssm_prefill(x, dt, a_log, cu, w, z=torch.zeros(T, 2, 32, dtype=bf), dims=d)
    with pytest.raises(ValueError, match="conv_w is required"):
        gdn.ssm_prefill(x, dt, a_log, cu, None, dims=d)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gdn.ssm_prefill(x.half(), dt, a_log, cu, w, dims=d)
    with pytest.raises(TypeError, match="conv_w must be"):
        gdn.ssm_prefill(x, dt, a_log, cu, w.float(), dims=d)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.ssm_prefill(x, dt, a_log, cu, torch.zeros(4, Cc, dtype=bf).T, dims=d)
    with pytest.raises(ValueError, match="pools hold 1 rows"):
        gdn.ssm_decode_step(x[:3], dt[:3], a_log, torch.zeros(4, 3, Cc, dtype=bf),
                            torch.zeros(1, 2, 64, 128), w, dims=d)
    with pytest.raises(ValueError, match="slot_idx holds"):
        gdn.ssm_decode_step(x[:3], dt[:3], a_log, torch.zeros(4, 3, Cc, dtype=bf),
                            torch.zeros(4, 2, 64, 128), w, slot_idx=torch.zeros(2).int(), dims=d)
    with pytest.raises(TypeError, match="S must be"):
        gdn.ssm_decode_step(x[:3], dt[:3], a_log, torch.zeros(4, 3, Cc, dtype=bf),
                            torch.zeros(4, 2, 64, 128).half(), w, dims=d)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        gdn.batch_tables(i(0), i(1), i(0), torch.zeros(1, 2).int(), i(1), i(0), 64, 1)
    with pytest.raises(ValueError, match="ctx_lens holds"):
        gdn.batch_tables(i(0), i(1, 2), i(0, 1), torch.zeros(2, 2).int(), i(1), i(0), 64, 3)
    with pytest.raises(ValueError, match="page_table holds 1 rows"):
        gdn.batch_tables(i(0, 0), i(1, 2), None, torch.zeros(1, 2).int(), i(1), i(0), 64, 3)
    with pytest.raises(ValueError, match="max_pages"):
        gdn.batch_tables(i(0, 0), i(1, 2), None, torch.zeros(4).int(), i(1), i(0), 64, 3)
    with pytest.raises(TypeError, match="new_lens must be"):
        gdn.batch_tables(i(0), torch.ones(1), i(0), torch.zeros(1, 2).int(), i(1), i(0), 64, 1)


def test_workspace_grows_with_the_batch(L):
    # one workspace, sized for the largest batch, takes every smaller one
    f = L.gdn_ssm_prefill_workspace_size
    for dims in (ref(), ref(num_heads=32, num_groups=16, head_dim=128), ref(num_groups=1),
                 ref(num_heads=4, num_groups=4), ref(num_heads=1024, num_groups=1, head_dim=128)):
        for dtype in (0, 1):
            for T in (0, 1, 127, 128, 5000, 40677, 65536, 1 << 20):
                for n0, n1 in ((1, 2), (2, 8), (8, 96), (96, 5000)):
                    assert f(dims, dtype, n0, T) <= f(dims, dtype, n1, T)
                for N in (1, 2, 8):
                    assert f(dims, dtype, N, T) <= f(dims, dtype, N, T + 129)
    big = (1 << 31) - 1
    assert f(ref(num_heads=1024, num_groups=1), 1, 1 << 25, 0) > 0
    assert f(ref(), 1, big, big) > f(ref(), 1, big, 0) > 0


def test_rows_of_x_have_the_layer_channels():
    d = gdn.SsmDims(2, 1)
    x, dt, a, w = torch.zeros(1, 7, d.channels), torch.zeros(7, 2), torch.zeros(2), torch.zeros(1)
    cu = torch.tensor([0, 7], dtype=torch.int32)
    for bad in (x, x[0, :, :-1], x[0, 0]):
        with pytest.raises(ValueError, match="x holds"):
            gdn.ssm_prefill(bad, dt, a, cu, w, dims=d)
        with pytest.raises(ValueError, match="x holds"):
            gdn.ssm_prefill_slots(bad, dt, a, cu, None, w, dims=d)
        with pytest.raises(ValueError, match="x holds"):
            gdn.ssm_decode_step(bad, dt, a, None, None, w, dims=d)
