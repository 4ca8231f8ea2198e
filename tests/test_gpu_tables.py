"""GPU checks of gdn_batch_tables against plain tables, and of a serving loop that uses it with
the layers that read its results."""
import numpy as np
import pytest
import torch

import gated_deltanet_layer_02_b200 as gdn
import ssm_util as U
from gated_deltanet_layer_02_b200 import inputs
from gpu_util import dev, dims_of, ensure_built

pytestmark = pytest.mark.gpu


def case(n, most_new, most_ctx, page, seed, spare=3):
    r = np.random.default_rng(seed)
    new = r.integers(0, most_new + 1, n)
    ctx = r.integers(0, most_ctx + 1, n)
    need = -(-(ctx + new) // page)
    held = -(-ctx // page)
    slots, width = n + 4, int(need.max()) + 2 if n else 3
    pages = int(need.sum()) + spare
    perm = r.permutation(pages)
    table = np.full((slots, width), -1, dtype=np.int32)
    slot = r.permutation(slots)[:n]
    at = 0
    for k in range(n):
        table[slot[k], :held[k]] = perm[at:at + held[k]]
        at += held[k]
    return ctx, new, slot, table, perm[at:]


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def run(ctx, new, slot, table, free, head, page, rows, status=None, **kw):
    ensure_built()
    t = i32(table)
    b = gdn.batch_tables(None if ctx is None else i32(ctx), i32(new),
                         None if slot is None else i32(slot), t, i32(free), i32([head]), page, rows,
                         dev_status=status, **kw)
    torch.cuda.synchronize()
    return b, t


def same(b, t, ref):
    cu, pos, where, head, table = ref
    assert b.cu_seqlens.tolist() == cu and b.positions.tolist() == pos
    assert b.slot_map.tolist() == where and b.free_head.tolist() == [head]
    np.testing.assert_array_equal(t.cpu().numpy(), table)


@pytest.mark.parametrize("pad", [0, 1, 1500])
@pytest.mark.parametrize("page", [1, 16, 48, 64])
@pytest.mark.parametrize("n,most_new,most_ctx", [(1, 1, 0), (1, 5000, 9), (7, 64, 200), (256, 1, 900),
                                                 (1023, 3, 70), (1024, 2, 5), (1025, 9, 300),
                                                 (4100, 2, 40), (3, 0, 10)])
def test_tables(n, most_new, most_ctx, page, pad):
    ctx, new, slot, table, free = case(n, most_new, most_ctx, page, seed=n + page)
    rows = int(new.sum()) + pad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b, t = run(ctx, new, slot, table, free, 2, page, rows, status)
    assert int(status.item()) == 0
    same(b, t, U.tables(ctx, new, slot, table, free, 2, page, rows))


def test_nothing_cached_and_identity_slots():
    new, page = [3, 0, 130, 64], 64
    table, free = np.full((4, 3), -1), np.arange(9)[::-1].copy()
    b, t = run(None, new, None, table, free, 1, page, 200)
    same(b, t, U.tables([0] * 4, new, range(4), table, free, 1, page, 200))


def test_no_requests_and_no_rows():
    b, t = run([], [], [], np.zeros((2, 3)), [4, 5], 1, 16, 5)
    assert b.cu_seqlens.tolist() == [0] and b.positions.tolist() == [-1] * 5
    assert b.slot_map.tolist() == [-1] * 5 and b.free_head.tolist() == [1]
    b, t = run([5], [0], [1], [[7, 7], [3, 9]], [4], 0, 16, 0)
    assert b.cu_seqlens.tolist() == [0, 0] and t.tolist() == [[7, 7], [3, 9]]


@pytest.mark.parametrize("n", [6, 2050])
def test_requests_that_break_a_rule_bring_no_token(n):
    page = 16
    ctx, new, slot, table, free = case(n, 40, 100, page, seed=5, spare=600)
    bad = {1: "slot", n - 1: "length", 3: "pages", 4: "position"}
    c, v, s = ctx.copy(), new.copy(), slot.copy()
    s[1] = len(table)
    v[n - 1] = -4
    v[3] = page * (table.shape[1] + 1)
    c[4], v[4] = 2 ** 31 - 5, 9
    rows = int(new.sum())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b, t = run(c, v, s, table, free, 0, page, rows, status)
    assert int(status.item()) == gdn.GDN_ERR_INVALID_ARG
    for k in bad:
        ctx[k] = new[k] = 0
    same(b, t, U.tables(ctx, new, slot, table, free, 0, page, rows))


@pytest.mark.parametrize("why", ["pages", "rows", "head", "negative head"])
def test_nothing_is_taken_when_the_batch_does_not_fit(why):
    page = 16
    ctx, new, slot, table, free = case(40, 30, 100, page, seed=6, spare=0)
    rows, head = int(new.sum()) + 9, 0
    if why == "pages":
        free = free[:-1]
    elif why == "rows":
        rows = int(new.sum()) - 1
    elif why == "head":
        head = len(free) + 1
    else:
        head = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b, t = run(ctx, new, slot, table, free, head, page, rows, status)
    want = gdn.GDN_ERR_PAGES if why == "pages" else gdn.GDN_ERR_INVALID_ARG
    assert int(status.item()) == want
    assert b.cu_seqlens.tolist() == [0] * 41 and set(b.positions.tolist()) == {-1}
    assert set(b.slot_map.tolist()) == {-1} and b.free_head.tolist() == [head]
    np.testing.assert_array_equal(t.cpu().numpy(), table)


def test_a_held_page_that_is_not_there():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b, t = run([20, 4], [3, 2], [0, 1], [[5, -1, -1], [6, -1, -1]], [8, 9], 0, 16, 5, status)
    assert int(status.item()) == gdn.GDN_ERR_INVALID_ARG
    assert b.slot_map.tolist() == [-1, -1, -1, 6 * 16 + 4, 6 * 16 + 5]
    assert b.positions.tolist() == [20, 21, 22, 4, 5]


def test_rows_past_32_bits():
    # a page number times a page size may pass 2^31
    b, _ = run([0], [3], [0], [[-1]], [2 ** 30], 0, 64, 3)
    assert b.slot_map.tolist() == [2 ** 36, 2 ** 36 + 1, 2 ** 36 + 2]


def test_serving_loop():
    """Prompts and then single tokens of three requests: the tables of every step are built on the
    device and feed a state space layer and a Gated DeltaNet layer on the same slots; the result is
    that of one call over the whole sequences."""
    ensure_built()
    shape, dtype = (4, 2, 64, 128), torch.bfloat16
    dims, steps, page = gdn.SsmDims(*shape), 3, 64
    prompt = [70, 1, 131]
    lens = [v + steps for v in prompt]
    i = U.inputs(*shape, lens, dtype, seed=30, init=False)
    w = inputs.custom(2, 4, 128, dtype, lengths=tuple(lens))
    gi = inputs.prefill_inputs(w, 3000)
    ref = U.layer(i, *shape)
    first = np.concatenate([[0], np.cumsum(lens)])
    slots, n_rows = 5, 5
    S = torch.zeros(slots, 4, 64, 128, device="cuda")
    c = torch.zeros(slots, 3, dims.channels, dtype=dtype, device="cuda")
    Sg = torch.zeros(slots, 4, 128, 128, device="cuda")
    cg = torch.zeros(slots, 3, w.channels, dtype=dtype, device="cuda")
    slot = i32([3, 0, 4])
    table = torch.full((slots, 4), -1, dtype=torch.int32, device="cuda")
    free, head = i32(np.arange(20)[::-1].copy()), i32([0])
    ctx, out, out_g = i32([0, 0, 0]), [[], [], []], [[], [], []]
    seen = [[], [], []]
    for step in range(steps + 1):
        count = prompt if step == 0 else [1, 1, 1]
        at = [0] * 3 if step == 0 else [prompt[k] + step - 1 for k in range(3)]
        rows = torch.tensor(np.concatenate([np.arange(first[k] + at[k], first[k] + at[k] + count[k])
                                            for k in range(3)]))
        new = i32(count)
        t = gdn.batch_tables(ctx, new, slot, table, free, head, page, sum(count))
        a = [dev(v[rows]) for v in (i["x"], i["dt"], i["z"])]
        kw = dict(conv_b=dev(i["conv_b"]), dt_bias=dev(i["dt_bias"]), D=dev(i["D"]), dims=dims)
        b = [dev(gi[k][rows]) for k in ("x", "beta", "g", "z")]
        if step == 0:
            o = gdn.ssm_prefill_slots(a[0], a[1], dev(i["a_log"]), t.cu_seqlens, S,
                                      dev(i["conv_w"]), slot_idx=slot, conv_pool=c, z=a[2], **kw)
            og = gdn.chunk_prefill_slots(b[0], b[1], b[2], t.cu_seqlens, Sg, slot_idx=slot,
                                         conv_pool=cg, conv_w=dev(gi["conv_w"]), z=b[3],
                                         norm_w=dev(gi["norm_w"]), dims=dims_of(w))
        else:
            o = gdn.ssm_decode_step(a[0], a[1], dev(i["a_log"]), c, S, dev(i["conv_w"]), z=a[2],
                                    slot_idx=slot, **kw)
            og = gdn.decode_step(b[0], b[1], b[2], cg, Sg, dev(gi["conv_w"]), z=b[3],
                                 norm_w=dev(gi["norm_w"]), slot_idx=slot, dims=dims_of(w))
        cu, pos, where = (v.tolist() for v in (t.cu_seqlens, t.positions, t.slot_map))
        for k in range(3):
            out[k].append(o[cu[k]:cu[k + 1]])
            out_g[k].append(og[cu[k]:cu[k + 1]])
            assert pos[cu[k]:cu[k + 1]] == list(range(at[k], at[k] + count[k]))
            seen[k] += where[cu[k]:cu[k + 1]]
        ctx, head = ctx + new, t.free_head
    got = torch.cat([torch.cat(v) for v in out])
    U.check_layer((got, S[slot.long()], c[slot.long()]), ref, dtype, "loop")
    flat = [r for v in seen for r in v]
    assert len(set(flat)) == len(flat)                      # no cache row is given twice
    assert int(head) == sum(-(-v // page) for v in lens)    # and no page too many
    for k in range(3):
        pages = table[int(slot[k])].tolist()
        assert seen[k] == [pages[q // page] * page + q % page for q in range(lens[k])]
    # the Gated DeltaNet layer on the same tables: that of one call over the whole sequences
    full, _, _ = gdn.chunk_prefill(dev(gi["x"]), dev(gi["beta"]), dev(gi["g"]),
                                   dev(gi["cu_seqlens"]), conv_w=dev(gi["conv_w"]),
                                   z=dev(gi["z"]), norm_w=dev(gi["norm_w"]), dims=dims_of(w))
    got_g = torch.cat([torch.cat(v) for v in out_g])
    err = (got_g.float() - full.float()).norm() / full.float().norm()
    assert float(err) <= 2e-2, float(err)   # the layer's own bar of the chunked bf16 path
