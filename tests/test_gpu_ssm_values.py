"""GPU checks of the state space layer's values at the ends of its inputs' ranges: magnitudes that
differ within a row, far negative gates, rates and steps at the ends of fp32, empty calls and
unusual sequence tables."""
import ctypes

import pytest
import torch

import gated_deltanet_layer_02_b200 as gdn
import ssm_bounds as SB
import ssm_util as U
from gpu_util import dev, ensure_built
from test_gpu_ssm import prefill

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


@DTYPES
@pytest.mark.parametrize("lens", [(127,), (128,), (130, 5)], ids=str)
def test_rate_past_fp32(lens, dtype):
    # exp(a_log) overflows: a token with a step forgets everything before it, one without a step
    # (softplus underflows) forgets nothing, and what lies behind the last token plays no part
    shape = (4, 2, 64, 128)
    i = U.inputs(*shape, lens, dtype, seed=50)
    i["a_log"][1] = 90.0
    i["dt"][3:9, 1] = -200.0
    i["dt"][lens[0] - 1, 1] = -200.0
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), dtype, f"rate {lens}")


@DTYPES
def test_rate_past_fp32_of_one_token(dtype):
    shape, B = (4, 2, 64, 128), 3
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (1,) * B, dtype, seed=51)
    i["a_log"][1] = 90.0
    i["dt"][1, 1] = -200.0
    ref = U.layer(i, *shape)
    ensure_built()
    S, c = dev(i["S0"]), dev(i["conv0"])
    o = gdn.ssm_decode_step(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), c, S, dev(i["conv_w"]),
                            conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]), D=dev(i["D"]),
                            z=dev(i["z"]), dims=dims)
    torch.cuda.synchronize()
    U.check(o, ref[0], ref[3], U.OUT_F32, "out", 2.0 ** -8 if dtype == BF else 0.0)
    U.check(S, ref[1], ref[4], U.STATE, "state")


@DTYPES
def test_gate_far_below_zero(dtype):
    # silu(z) = z / (1 + exp(-z)) keeps its relative precision down to where it underflows, and is
    # zero below
    shape = (4, 2, 64, 128)
    i = U.inputs(*shape, (70, 9), dtype, seed=52)
    values = [-30.0, -43.5, -50.0, -60.0, -88.0, -100.0, -1e10, -1e30, torch.finfo(BF).min]
    z = i["z"].view(-1)
    for k, v in enumerate(values):
        z[k::16] = v
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), dtype, "gate")


@pytest.mark.parametrize("what", ["x", "B", "C"])
def test_conv_output_far_below_zero(what):
    # silu is zero at -200 and below: the same bits whatever the value
    shape = (4, 2, 64, 128)
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (150,), BF, seed=53, init=False)
    c = {"x": 70, "B": 4 * 64 + 5, "C": 4 * 64 + 2 * 128 + 5}[what]
    i["conv_w"][c] = torch.tensor([0.0, 0.0, 0.0, 1.0])
    got = []
    for v in (-200.0, -1e30):
        i["x"][17, c] = i["x"][131, c] = v
        got.append(prefill(i, dims))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    U.check_layer((got[1][0], None, None), U.layer(dict(i, x=i["x"].clamp(min=-200.0)), *shape), BF,
                  what)


def one_large(mag, L, what="x", seed=40):
    """A prompt with slow decays, in which token 10 has one value of about `mag` among ones."""
    i = U.inputs(2, 1, 64, 128, (L,), BF, seed, init=False, gate=False, direct=False)
    i["a_log"].fill_(-3.0)
    c = 5 if what == "x" else 2 * 64 + 7
    i["conv_w"][c] = torch.tensor([0.0, 0.0, 0.0, 1.0])
    i["x"][10, c] = mag
    if what == "B":  # where C is zero: no output shows the value itself
        i["conv_w"][c + 128], i["conv_b"][c + 128] = 0.0, 0.0
    return i


@pytest.mark.parametrize("L", [128, 300])
@pytest.mark.parametrize("what", ["x", "B"])
@pytest.mark.parametrize("e", [19, 20, 22])
def test_one_large_value_leaves_the_others(e, what, L):
    # 2^22 times as large as the others of its row: they keep the ordinary bound
    i = one_large(2.0 ** e, L, what)
    U.check_layer(prefill(i, gdn.SsmDims(2, 1, 64, 128)), U.layer(i, 2, 1, 64, 128), BF,
                  f"{what} 2^{e}")


@pytest.mark.parametrize("what", ["x", "B"])
@pytest.mark.parametrize("e", [0, 24, 30])
def test_one_large_value_within_the_bound_of_fp16_operands(e, what):
    i = one_large(2.0 ** e, 128, what, seed=41)
    o, S, _ = prefill(i, gdn.SsmDims(2, 1, 64, 128))
    out, SN, b_out, b_SN = SB.chunk_bounds(i, 2, 1, 64, 128)
    assert SB.worst(o, out, b_out) <= 1.0
    assert SB.worst(S, SN, b_SN) <= 1.0


@DTYPES
@pytest.mark.parametrize("cu", [(101, 203, 0, 101), (0, 50, -1, 101, 203, 203),
                                (0, 50, 50, 2 ** 31 - 1, 50, 203)], ids=str)
def test_bad_entries_cost_no_other_sequence_its_rows(cu, dtype):
    # entries out of order or outside the rows: their sequences count as empty, the others are
    # computed like any other
    shape, T, N = (2, 1, 64, 128), 203, len(cu) - 1
    good = [n for n in range(N) if 0 <= cu[n] <= cu[n + 1] <= T]
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (T,), dtype, seed=55, init=False)
    S0 = 0.1 * torch.randn(N, 2, 64, 128, generator=torch.Generator().manual_seed(4))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ensure_built()
    ws = torch.full((gdn.ssm_prefill_workspace_size(N, T, dtype, dims),), 0x7f, dtype=torch.uint8,
                    device="cuda")
    o, S, c = gdn.ssm_prefill(
        dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), torch.tensor(cu, dtype=torch.int32).cuda(),
        dev(i["conv_w"]), conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]), D=dev(i["D"]),
        z=dev(i["z"]), S0=dev(S0), dims=dims, dev_status=status, workspace=ws)
    torch.cuda.synchronize()
    assert int(status.item()) == gdn.GDN_ERR_INVALID_ARG
    for n in range(N):
        if n not in good:
            assert torch.equal(S[n].cpu(), S0[n])
            continue
        rows = slice(cu[n], cu[n + 1])
        j = dict(i, x=i["x"][rows], dt=i["dt"][rows], z=i["z"][rows], S0=S0[n:n + 1],
                 cu=torch.tensor([0, cu[n + 1] - cu[n]]))
        U.check_layer((o[rows], S[n:n + 1], c[n:n + 1]), U.layer(j, *shape), dtype, f"sequence {n}")


def spread(shape, lens, seed, e=12):
    """Inputs whose channels of x, B and C, and elements of the state, differ by up to 2^(2 e)."""
    H, G, P, N = shape
    i = U.inputs(*shape, lens, BF, seed=seed)
    gen = torch.Generator().manual_seed(seed)
    i["x"] = (i["x"].float() * 2.0 ** torch.randint(-e, e + 1, (1, H * P + 2 * G * N),
                                                    generator=gen)).to(BF)
    i["S0"] = i["S0"] * 2.0 ** torch.randint(-e, e + 1, (1, H, P, N), generator=gen)
    i["conv0"], i["conv_b"] = None, None
    return i


@pytest.mark.parametrize("shape", [(4, 2, 64, 128), (2, 1, 128, 64)], ids=str)
@pytest.mark.parametrize("lens", [(1,), (3,), (5, 0, 2), (40, 128)], ids=str)
def test_channels_of_other_magnitudes(lens, shape):
    # short sequences too, in which no errors average out
    i = spread(shape, lens, seed=60 + len(lens))
    o, S, _ = prefill(i, gdn.SsmDims(*shape))
    out, SN, b_out, b_SN = SB.chunk_bounds(i, *shape)
    assert SB.worst(o, out, b_out) <= 1.0
    assert SB.worst(S, SN, b_SN) <= 1.0


def exact_conv(shape, lens, seed):
    """Inputs whose conv is its last tap alone, with slow decays."""
    i = U.inputs(*shape, lens, BF, seed=seed, bias=False)
    i["conv_w"] = torch.tensor([0.0, 0.0, 0.0, 1.0], dtype=BF).repeat(i["conv_w"].shape[0], 1)
    i["conv0"] = None
    i["x"] = i["x"].clamp(-7.0, 7.0)
    i["a_log"].fill_(-6.0)
    return i


@pytest.mark.parametrize("shape", [(4, 2, 64, 128), (2, 1, 128, 64)], ids=str)
@pytest.mark.parametrize("lens", [(1,), (2,), (5, 0, 3, 1)], ids=str)
def test_both_parts_of_the_state_factors_count(lens, shape):
    i = exact_conv(shape, lens, seed=70 + len(lens))
    o, S, _ = prefill(i, gdn.SsmDims(*shape))
    out, SN, b_out, b_SN = SB.chunk_bounds(i, *shape, SB.TIGHT_OUT, SB.TIGHT_STATE)
    assert SB.worst(o, out, b_out) <= 1.0
    assert SB.worst(S, SN, b_SN) <= 1.0


def test_both_parts_count_in_a_state_that_segments_hand_on():
    # three tokens at the start of a sequence of 16 chunks; the others bring nothing.  Each chunk's
    # decay and the product with it are off by 2^-23 and 2^-24: with 16 of them below 2^-18 more
    shape, T = (2, 1, 64, 128), 2000
    i = exact_conv(shape, (T,), seed=75)
    i["x"][3:] = 0
    o, S, _ = prefill(i, gdn.SsmDims(*shape))
    _, SN, _, _, scale = U.layer(i, *shape)
    assert SB.worst(S, SN, (SB.TIGHT_STATE + 2.0 ** -18) * scale + 2.0 ** -100) <= 1.0


@pytest.mark.parametrize("lens", [(100,), (128, 40), (700,)], ids=str)
@DTYPES
def test_tokens_without_a_step_leave_the_state_whatever_their_rows_hold(dtype, lens):
    # a padded batch that masks its last tokens by their steps: 0 times a row of 1e30 is nothing
    shape, pad = (4, 2, 64, 128), 20
    i = U.inputs(*shape, lens, dtype, seed=57)
    for e in i["cu"][1:].tolist():
        i["dt"][e - pad:e] = -1e4
        i["x"][e - pad:e] *= 1e30
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), dtype, "masked")


@DTYPES
@pytest.mark.parametrize("first", [1, 2, 150])
def test_rows_before_the_first_sequence_stay(first, dtype):
    shape, T = (2, 1, 64, 128), 290
    i = U.inputs(*shape, (T - first,), dtype, seed=58)
    want = prefill(i, gdn.SsmDims(*shape))
    pad = lambda t: torch.cat([torch.full((first, *t.shape[1:]), float("nan"), dtype=t.dtype), t])  # noqa: E731
    j = dict(i, x=pad(i["x"]), dt=pad(i["dt"]), z=pad(i["z"]), cu=i["cu"] + first)
    out = torch.full((T, 2, 64), 7.0, dtype=dtype, device="cuda")
    got = prefill(j, gdn.SsmDims(*shape), out=out)
    assert torch.all(out[:first] == 7.0)
    for a, b in zip((out[first:], got[1], got[2]), want):
        assert torch.equal(a, b)
