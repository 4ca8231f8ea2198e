"""GPU parity of the selective state space layer (packed prefill, slots, single tokens) against
its definition in fp64, at the lengths, shapes and states where it can go wrong."""
import numpy as np
import pytest
import torch

import gated_deltanet_layer_02_b200 as gdn
import ssm_util as U
from gpu_util import dev, ensure_built

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(2, 1, 64, 128), (4, 2, 128, 128), (3, 1, 64, 64), (6, 2, 128, 64), (8, 8, 64, 128)]
LENGTHS = [(1,), (37,), (128,), (129,), (5, 0, 129, 64, 1), (256, 300), (2, 3, 1, 0, 0, 4),
           (1000,), (0,)]


def prefill(i, dims, **kw):
    ensure_built()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = gdn.ssm_prefill(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), dev(i["cu"]), dev(i["conv_w"]),
                        conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]), D=dev(i["D"]),
                        z=dev(i["z"]), S0=dev(i["S0"]), conv0=dev(i["conv0"]), dims=dims,
                        dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return r


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_prefill(shape, lens, dtype):
    i = U.inputs(*shape, lens, dtype, seed=100 + sum(lens))
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), dtype, f"{shape} {lens}")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [64, 128])
def test_prefill_many_heads_and_sequences(N, dtype):
    # enough (sequence, head) pairs for a CTA to take 64 rows of a state in fp32
    shape, lens = (32, 4, 64, N), (3, 20, 1, 0, 17, 33, 2, 1, 40, 5)
    i = U.inputs(*shape, lens, dtype, seed=6)
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), dtype, f"many {N}")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off", ["init", "gate", "bias", "direct"])
def test_prefill_without_an_optional_part(off, dtype):
    shape, lens = (4, 2, 64, 128), (130, 3)
    i = U.inputs(*shape, lens, dtype, seed=7, **{off: False})
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), dtype, off)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", ["large", "tiny", "no decay", "strong decay", "clamped step",
                                  "mixed magnitudes"])
def test_prefill_extremes(case, dtype):
    shape, lens = (4, 2, 64, 128), (200, 70)
    i = U.inputs(*shape, lens, dtype, seed=11,
                 std={"large": 64.0, "tiny": 2.0 ** -20}.get(case, 1.0))
    kw = {}
    if case == "no decay":
        i["a_log"].fill_(-40.0)
    elif case == "strong decay":
        i["a_log"].fill_(5.0)
    elif case == "clamped step":
        kw = dict(dt_min=0.05, dt_max=0.1)
    elif case == "mixed magnitudes":  # rows and channels whose sizes differ by 2^24
        i["x"] = (i["x"].float() * 2.0 ** torch.randint(-12, 13, (270, 1), generator=torch.
                                                        Generator().manual_seed(3))).to(dtype)
    U.check_layer(prefill(i, gdn.SsmDims(*shape, **kw)), U.layer(i, *shape, **kw), dtype, case)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_long_sequence(dtype):
    # several segments of a sequence, the last one ragged, beside a short one
    shape, lens = (2, 1, 64, 128), (4111, 9)
    i = U.inputs(*shape, lens, dtype, seed=12)
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), dtype, "long")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_prefill_in_place_states_and_no_states(dtype):
    shape, lens = (4, 2, 64, 128), (130, 0, 2, 65)
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, dtype, seed=13)
    out, SN, convN = prefill(i, dims)
    S, c = dev(i["S0"]).clone(), dev(i["conv0"]).clone()
    o2, S2, c2 = gdn.ssm_prefill(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), dev(i["cu"]),
                                 dev(i["conv_w"]), conv_b=dev(i["conv_b"]),
                                 dt_bias=dev(i["dt_bias"]), D=dev(i["D"]), z=dev(i["z"]), S0=S,
                                 SN=S, conv0=c, convN=c, dims=dims)
    o3, S3, c3 = prefill(i, dims, want_state=False)
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(S2, SN) and torch.equal(c2, convN)
    assert torch.equal(o3, out) and S3 is None and c3 is None


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_split_calls_continue_one_another(dtype):
    # the states of one call carry on in the next, cut anywhere
    shape, L, cut = (2, 1, 64, 128), 300, 171
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (L,), dtype, seed=14)
    ref = U.layer(i, *shape)
    a = dict(i, x=i["x"][:cut], dt=i["dt"][:cut], z=i["z"][:cut], cu=torch.tensor([0, cut]).int())
    o1, S1, c1 = prefill(a, dims)
    b = dict(i, x=i["x"][cut:], dt=i["dt"][cut:], z=i["z"][cut:],
             cu=torch.tensor([0, L - cut]).int(), S0=S1.cpu(), conv0=c1.cpu())
    o2, S2, c2 = prefill(b, dims)
    # the state is handed over in fp32, its error does not grow in the second part
    U.check_layer((torch.cat([o1, o2]), S2, c2), ref, dtype, "split")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_slots_equal_the_dense_call(dtype):
    shape, lens, slots, rows = (4, 2, 64, 128), (130, 0, 5, 257), [4, 1, 0, 2], 6
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, dtype, seed=15)
    out, SN, convN = prefill(i, dims)
    S = torch.full((rows, 4, 64, 128), 3.0, device="cuda")
    c = torch.full((rows, 3, dims.channels), 5.0, dtype=dtype, device="cuda")
    slot = torch.tensor(slots, dtype=torch.int32, device="cuda")
    S[slot.long()], c[slot.long()] = dev(i["S0"]), dev(i["conv0"])
    S_was, c_was = S.clone(), c.clone()
    args = (dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), dev(i["cu"]))
    kw = dict(conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]), D=dev(i["D"]), z=dev(i["z"]),
              dims=dims)
    o = gdn.ssm_prefill_slots(*args, S, dev(i["conv_w"]), slot_idx=slot, conv_pool=c, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, out)
    assert torch.equal(S[slot.long()], SN) and torch.equal(c[slot.long()], convN)
    for r in (3, 5):
        assert torch.all(S[r] == 3.0) and torch.all(c[r] == 5.0)
    # slots outside the pool: zero states, nothing kept, reported; the others as before
    bad = torch.tensor([4, -1, 6, 2], dtype=torch.int32, device="cuda")
    S, c = S_was.clone(), c_was.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = gdn.ssm_prefill_slots(*args, S, dev(i["conv_w"]), slot_idx=bad, conv_pool=c,
                              dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == gdn.GDN_ERR_INVALID_ARG
    zero = dict(i, S0=i["S0"].clone(), conv0=i["conv0"].clone())
    for n in (1, 2):
        zero["S0"][n], zero["conv0"][n] = 0, 0
    o0, _, _ = prefill(zero, dims)
    assert torch.equal(o, o0)
    assert torch.equal(S[4], SN[0]) and torch.equal(S[2], SN[3])
    for r in (0, 1, 3, 5):
        assert torch.equal(S[r], S_was[r]) and torch.equal(c[r], c_was[r])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_behind_the_last_sequence_stay(dtype):
    shape, lens, pad = (2, 1, 64, 128), (70, 131), 150
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens + (pad,), dtype, seed=16)
    i["x"][-pad:] = float("nan")
    i["dt"][-pad:] = float("nan")
    i["z"][-pad:] = float("nan")
    i.update(cu=i["cu"][:-1], S0=i["S0"][:-1], conv0=i["conv0"][:-1])
    out = torch.full((sum(lens) + pad, 2, 64), 7.0, dtype=dtype, device="cuda")
    o, SN, c = prefill(i, dims, out=out)
    assert torch.all(o[-pad:] == 7.0)
    j = dict(i, x=i["x"][:-pad], dt=i["dt"][:-pad], z=i["z"][:-pad])
    U.check_layer((o[:-pad], SN, c), U.layer(j, *shape), dtype, "padded batch")


def test_bad_cu_seqlens_are_reported_and_read_nothing_outside():
    # entries out of order or past num_tokens: those sequences count as empty
    shape, T = (2, 1, 64, 128), 40
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (T,), BF, seed=17)
    for cu in ([0, 30, 20, 40], [0, 10, 90, 40], [-5, 10, 20, 40]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        S0 = torch.randn(3, 2, 64, 128, device="cuda")
        out, SN, _ = gdn.ssm_prefill(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]),
                                     torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                     dev(i["conv_w"]), S0=S0, dims=dims, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == gdn.GDN_ERR_INVALID_ARG
        bad = [n for n in range(3) if cu[n] < 0 or cu[n + 1] < cu[n] or cu[n + 1] > T]
        for n in bad:
            assert torch.equal(SN[n], S0[n])


@pytest.mark.parametrize("state", [F32, BF], ids=["state32", "state16"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + [(16, 1, 64, 128), (10, 2, 128, 64)], ids=str)
def test_decode(shape, dtype, state):
    H, G, P, N = shape
    B, rows = 5, 9
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (1,) * B, dtype, seed=18)
    slot = torch.tensor([8, 0, 3, 7, 2], dtype=torch.int32)
    S = (0.1 * torch.randn(rows, H, P, N, generator=torch.Generator().manual_seed(1))).to(state)
    c = torch.randn(rows, 3, dims.channels, generator=torch.Generator().manual_seed(2)).to(dtype)
    ref = U.layer(dict(i, S0=S[slot.long()], conv0=c[slot.long()]), *shape)
    Sd, cd = S.cuda(), c.cuda()
    ensure_built()
    o = gdn.ssm_decode_step(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), cd, Sd, dev(i["conv_w"]),
                            conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]), D=dev(i["D"]),
                            z=dev(i["z"]), slot_idx=dev(slot), dims=dims)
    torch.cuda.synchronize()
    at = slot.long()
    # fp32 throughout: the outputs are as exact as the fp32 path's, before their own rounding
    half = 2.0 ** -8
    U.check(o, ref[0], ref[3], U.OUT_F32, "out", half if dtype == BF else 0.0)
    U.check(Sd[at.cuda()], ref[1], ref[4], U.STATE, "state", half if state == BF else 0.0)
    np.testing.assert_array_equal(U.f64(cd[at.cuda()]), ref[2])
    for r in (1, 4, 5, 6):
        assert torch.equal(Sd[r].cpu(), S[r]) and torch.equal(cd[r].cpu(), c[r])
    # a slot outside the pool is skipped and reported
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    S2, c2 = S.cuda(), c.cuda()
    out = torch.full((B, H, P), 7.0, dtype=dtype, device="cuda")
    bad = torch.tensor([8, 9, 3, -1, 2], dtype=torch.int32, device="cuda")
    gdn.ssm_decode_step(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), c2, S2, dev(i["conv_w"]),
                        conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]), D=dev(i["D"]),
                        z=dev(i["z"]), slot_idx=bad, dims=dims, out=out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == gdn.GDN_ERR_INVALID_ARG
    for b in range(B):
        if b in (1, 3):
            assert torch.all(out[b] == 7.0)
        else:
            assert torch.equal(out[b], o[b]) and torch.equal(S2[slot[b]], Sd[slot[b]])
    for r in (0, 7):
        assert torch.equal(S2[r].cpu(), S[r]) and torch.equal(c2[r].cpu(), c[r])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_empty_calls(dtype):
    ensure_built()
    dims = gdn.SsmDims(2, 1)
    e = lambda *s, t=dtype: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    w, a_log = torch.ones(dims.channels, 4, dtype=dtype, device="cuda"), torch.zeros(2).cuda()
    out, SN, c = gdn.ssm_prefill(e(0, dims.channels), e(0, 2, t=F32), a_log,
                                 torch.zeros(1, dtype=torch.int32, device="cuda"), w, dims=dims)
    assert out.shape == (0, 2, 64) and SN.shape[0] == 0 and c.shape[0] == 0
    o = gdn.ssm_decode_step(e(0, dims.channels), e(0, 2, t=F32), a_log, e(1, 3, dims.channels),
                            e(1, 2, 64, 128, t=F32), w, dims=dims)
    assert o.shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_captured_and_replayed_on_another_stream(dtype):
    shape, lens = (4, 2, 64, 128), (300, 40)
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, dtype, seed=19)
    out, SN, convN = prefill(i, dims)
    d = {k: dev(v) for k, v in i.items()}
    slot = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    S, c = torch.empty_like(SN), torch.empty_like(convN)
    kw = dict(conv_b=d["conv_b"], dt_bias=d["dt_bias"], D=d["D"], dims=dims)

    def step():
        o = gdn.ssm_prefill_slots(d["x"], d["dt"], d["a_log"], d["cu"], S, d["conv_w"],
                                  slot_idx=slot, conv_pool=c, z=d["z"], **kw)
        q = gdn.ssm_decode_step(d["x"][:2], d["dt"][:2], d["a_log"], c, S, d["conv_w"],
                                slot_idx=slot, **kw)
        return o, q

    S[slot.long()], c[slot.long()] = d["S0"], d["conv0"]
    o1, q1 = step()
    S1, c1 = S.clone(), c.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o2, q2 = step()
        for _ in range(3):
            S[slot.long()], c[slot.long()] = d["S0"], d["conv0"]
            o2.zero_()
            g.replay()
    s.synchronize()
    assert torch.equal(o1, out) and torch.equal(o2, o1) and torch.equal(q2, q1)
    assert torch.equal(S, S1) and torch.equal(c, c1)


def test_two_calls_at_once():
    shape = (4, 2, 64, 128)
    dims = gdn.SsmDims(*shape)
    work = [U.inputs(*shape, lens, BF, seed=20 + k) for k, lens in enumerate([(700,), (90, 500)])]
    alone = [prefill(i, dims) for i in work]
    d = [{k: dev(v) for k, v in i.items()} for i in work]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in work], [[], []]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                e = d[k]
                got[k].append(gdn.ssm_prefill(e["x"], e["dt"], e["a_log"], e["cu"], e["conv_w"],
                                              conv_b=e["conv_b"], dt_bias=e["dt_bias"], D=e["D"],
                                              z=e["z"], S0=e["S0"], conv0=e["conv0"], dims=dims))
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(r, alone[k]))


def _isolated(clean, broken, cu, seq, t, head, width):
    """`broken` has a non-finite input at token t of sequence `seq` and head `head`: the head's
    outputs from there on (`width` channels of them) and its state are not finite, and everything
    else has the bits of `clean`."""
    at, end = int(cu[seq]) + t, int(cu[seq + 1])
    ch = slice(0, width)
    assert not torch.any(torch.isfinite(broken[0][at:end, head, ch].float()))
    assert not torch.any(torch.isfinite(broken[1][seq, head, ch]))
    keep = torch.ones_like(clean[0], dtype=torch.bool)
    keep[at:end, head, ch] = False
    assert torch.equal(broken[0][keep], clean[0][keep])
    keep = torch.ones_like(clean[1], dtype=torch.bool)
    keep[seq, head, ch] = False
    assert torch.equal(broken[1][keep], clean[1][keep])


@pytest.mark.parametrize("t", [0, 37, 130, 299])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_nan_step_reaches_its_head_from_its_token_on(dtype, t):
    shape, lens = (4, 2, 128, 128), (50, 300, 60)
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, dtype, seed=31)
    clean = prefill(i, dims)
    i["dt"][50 + t, 2] = float("nan")
    _isolated(clean, prefill(i, dims), i["cu"], 1, t, 2, 128)


def test_nan_step_of_one_token():
    shape, B = (4, 2, 64, 128), 3
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (1,) * B, BF, seed=32)
    ensure_built()

    def step():
        S, c = dev(i["S0"]), dev(i["conv0"])
        o = gdn.ssm_decode_step(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), c, S, dev(i["conv_w"]),
                                dims=dims)
        return o, S

    clean = step()
    i["dt"][1, 3] = float("nan")
    _isolated(clean, step(), i["cu"], 1, 0, 3, 64)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("t", [1, 100, 128, 298])
def test_non_finite_x_reaches_its_channels_from_its_token_on(t, value):
    # one channel of x of head 2 (its second 64 of 128); the chunked form makes the 64 NaN
    shape, lens = (4, 2, 128, 128), (50, 300, 60)
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, BF, seed=33)
    i["conv_w"][2 * 128 + 70] = 1.0  # every tap passes it on
    clean = prefill(i, dims)
    i["x"][50 + t, 2 * 128 + 70] = value
    o, S, _ = prefill(i, dims)
    at, end, ch = 50 + t, 350, slice(64, 128)
    assert not torch.any(torch.isfinite(o[at:end, 2, ch].float()))
    assert not torch.any(torch.isfinite(S[1, 2, ch]))
    for got, was in ((o, clean[0]), (S, clean[1])):
        keep = torch.ones_like(was, dtype=torch.bool)
        if got is o:
            keep[at:end, 2, ch] = False
        else:
            keep[1, 2, ch] = False
        assert torch.equal(got[keep], was[keep])


@pytest.mark.parametrize("what", ["B", "C"])
def test_non_finite_b_or_c_reaches_its_group_from_its_token_on(what):
    shape, lens, t = (4, 2, 64, 128), (50, 300, 60), 140
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, BF, seed=34)
    c = 4 * 64 + (0 if what == "B" else 2 * 128) + 128 + 5  # of group 1: heads 2 and 3
    i["conv_w"][c] = 1.0
    clean = prefill(i, dims)
    i["x"][50 + t, c] = float("inf")
    o, S, _ = prefill(i, dims)
    end = 350 if what == "B" else 50 + t + 4  # C: as long as the conv sees it
    assert not torch.any(torch.isfinite(o[50 + t:end, 2:].float()))
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[50 + t:end, 2:] = False
    assert torch.equal(o[keep], clean[0][keep])
    keep = torch.ones_like(S, dtype=torch.bool)
    if what == "B":
        assert not torch.any(torch.isfinite(S[1, 2:]))
        keep[1, 2:] = False
    assert torch.equal(S[keep], clean[1][keep])


@pytest.mark.parametrize("lens", [
    (300,) + (5, 0, 140) * 10 + (257,),          # 32 sequences, the most taken longest first
    (129,) + (0, 7, 260) * 11,                   # 34
    (3,) * 100 + (400,) + (0, 1) * 30 + (130,),  # 162: more than are looked at at once
], ids=["32", "34", "162"])
def test_prefill_of_many_sequences_in_segments(lens):
    shape = (2, 1, 64, 128)
    i = U.inputs(*shape, lens, BF, seed=35)
    U.check_layer(prefill(i, gdn.SsmDims(*shape)), U.layer(i, *shape), BF, str(len(lens)))


def test_workspace_of_a_larger_batch():
    # sized once for the largest batch, used for others, with what those before left in it
    shape = (4, 2, 64, 128)
    dims = gdn.SsmDims(*shape)
    ensure_built()
    ws = torch.full((gdn.ssm_prefill_workspace_size(9, 1500, BF, dims),), 0x7f,
                    dtype=torch.uint8, device="cuda")
    for lens in ((1500,), (700, 0, 3, 130, 1, 1, 1, 600, 64), (129,)):
        i = U.inputs(*shape, lens, BF, seed=36)
        got, want = prefill(i, dims, workspace=ws), prefill(i, dims)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("batch", [1, 40, 83, 150])
@pytest.mark.parametrize("shape", [(48, 1, 64, 128), (24, 2, 64, 64), (7, 1, 128, 128)], ids=str)
def test_decode_of_other_batches_has_the_same_bits(shape, batch):
    # how many CTAs share a group goes by the batch; the sums of a row do not
    H, G, P, N = shape
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, (1,) * batch, BF, seed=37)
    S, c = dev(i["S0"]), dev(i["conv0"])
    ensure_built()

    def step(n, k):  # sequences n .. n + k - 1
        s, h = S[n:n + k].clone(), c[n:n + k].clone()
        o = gdn.ssm_decode_step(dev(i["x"][n:n + k]), dev(i["dt"][n:n + k]), dev(i["a_log"]), h, s,
                                dev(i["conv_w"]), conv_b=dev(i["conv_b"]), D=dev(i["D"]),
                                z=dev(i["z"][n:n + k]), dims=dims)
        return o, s, h

    o, s, h = step(0, batch)
    for n in sorted({0, batch // 2, batch - 1}):
        for got, one in zip((o, s, h), step(n, 1)):
            assert torch.equal(got[n:n + 1], one)


@pytest.mark.parametrize("off", [8, 16], ids=["16 bytes", "32 bytes"])
def test_output_aligned_to_16_bytes(off):
    # outputs leave 32 bytes at a time where their address allows it, 16 else: the same values
    shape, lens = (4, 2, 64, 128), (130, 3, 200)
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, BF, seed=38)
    want = prefill(i, dims)[0]
    buf = torch.full((want.numel() + 2 * off,), 7.0, dtype=BF, device="cuda")
    out = buf[off:off + want.numel()].view_as(want)
    prefill(i, dims, out=out)
    assert torch.equal(out, want)
    assert torch.all(buf[:off] == 7.0) and torch.all(buf[-off:] == 7.0)


@pytest.mark.parametrize("off", [8, 16], ids=["16 bytes", "32 bytes"])
def test_gate_aligned_to_16_bytes(off):
    shape, lens = (4, 2, 64, 128), (130, 3, 200)
    dims = gdn.SsmDims(*shape)
    i = U.inputs(*shape, lens, BF, seed=38)
    want = prefill(i, dims)[0]
    z = dev(i["z"])
    buf = torch.full((z.numel() + 2 * off,), float("nan"), dtype=BF, device="cuda")
    at = buf[off:off + z.numel()].view_as(z)
    at.copy_(z)
    got = gdn.ssm_prefill(dev(i["x"]), dev(i["dt"]), dev(i["a_log"]), dev(i["cu"]),
                          dev(i["conv_w"]), conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]),
                          D=dev(i["D"]), z=at, S0=dev(i["S0"]), conv0=dev(i["conv0"]), dims=dims)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
