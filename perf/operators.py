"""Cases, plain forms and exact values of the state space operators and of the batch tables.

Three operators, each with the plain form that its kernels are compared with:

  prefill  selective state space scan of packed prompts with its causal convolution (ssm_prefill)
  decode   the same layer for one token of each of B sequences, states in a slot pool
           (ssm_decode_step)
  tables   cu_seqlens, positions, page table and slot map of a batch, from the requests' lengths
           (batch_tables)

The layer, per token t of a sequence, head h (group g = h / (H / G)), with row [x | B | C] of
H P + 2 G N channels:
  u        = silu(sum_i w[c, i] row_{t-3+i}[c] + b[c])             (depthwise, causal, width 4)
  delta    = min(max(softplus(dt[t, h] + dt_bias[h]), dt_min), dt_max)
  S_t      = exp(-exp(a_log[h]) delta) S_{t-1} + delta x_t B_t^T   ([P, N] per head)
  y_t      = S_t C_t + D[h] x_t
  out_t    = y_t silu(z_t)

The tables, for request n with ctx[n] tokens in the cache and new[n] to come, whose pages are
named by row slot[n] of the page table: it takes the pages it lacks from the free list, in the
order of the requests; token j of it has position ctx[n] + j and goes to row
page_table[slot[n]][position / page] page + position % page of the cache.
"""
import math
import random

import torch

own = False

CONV = 4       # conv width
CHUNK = 128    # chunk of the plain form of the scan


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a short chat prompt on an idle server: latency counts
        dict(name="prompt_37", op="prefill", dtype="bf16", H=64, G=8, P=64, N=128, tokens=37,
             seqs=1, spread=0.0, init=False, gate=True),
        # one prompt at the layer shape of this repository (16 key heads, 32 value heads of 128)
        dict(name="prompt_4096", op="prefill", dtype="bf16", H=32, G=16, P=128, N=128,
             tokens=4096, seqs=1, spread=0.0, init=False, gate=True),
        # the packed batch of this repository: 8 sequences, 40,677 tokens, states carried on
        dict(name="packed_8", op="prefill", dtype="bf16", H=64, G=1, P=64, N=128, tokens=40677,
             seqs=8, spread=0.8, init=True, gate=True),
        # a long document in one call
        dict(name="document_65536", op="prefill", dtype="bf16", H=64, G=8, P=64, N=128,
             tokens=65536, seqs=1, spread=0.0, init=False, gate=True),
        # many short prompts of a batch of requests, half the state width
        dict(name="packed_96_short", op="prefill", dtype="bf16", H=24, G=2, P=64, N=64,
             tokens=5003, seqs=96, spread=0.9, init=True, gate=False),
        # fp32 activations, as a reference run or an evaluation has them
        dict(name="f32_1021", op="prefill", dtype="f32", H=4, G=2, P=128, N=128, tokens=1021,
             seqs=3, spread=0.5, init=True, gate=True),
        # one user's next token
        dict(name="token_1", op="decode", dtype="bf16", state="f32", H=64, G=8, P=64, N=128,
             batch=1, gate=True),
        # the decode batch of this repository: 256 sequences at its layer shape
        dict(name="token_256", op="decode", dtype="bf16", state="f32", H=32, G=16, P=128, N=128,
             batch=256, gate=True),
        # a ragged batch with the state kept in 16 bits
        dict(name="token_83_bf16_state", op="decode", dtype="bf16", state="bf16", H=48, G=1, P=64,
             N=128, batch=83, gate=True),
        # tables of a decode step: one new token for each of 256 requests
        dict(name="tables_decode_256", op="tables", requests=256, most_new=1, most_ctx=8192,
             page=64, pad=0),
        # tables of the packed batch of this repository: 8 prompts with nothing cached
        dict(name="tables_prompts_8", op="tables", requests=8, most_new=8192, most_ctx=0, page=64,
             pad=283),
        # a large serving step: chunks of prompts and single tokens of 4096 requests
        dict(name="tables_4096", op="tables", requests=4096, most_new=128, most_ctx=16384, page=16,
             pad=1000),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    G = rng.choice([1, 2, 4, 8])
    per = rng.choice([1, 2, 3, 4, 8])
    H = G * per
    if H > 64:
        H = G * 4
    return H, G, rng.choice([64, 64, 128]), rng.choice([128, 128, 64])


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "tables"])
    if op == "prefill":
        H, G, P, N = _heads(rng)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        tokens = _spread(rng, 1, 2000 if dtype == "f32" else 20000)
        seqs = min(_spread(rng, 1, 64), tokens)
        return dict(op=op, dtype=dtype, H=H, G=G, P=P, N=N, tokens=tokens, seqs=seqs,
                    spread=round(rng.uniform(0.0, 1.0), 2), init=rng.random() < 0.5,
                    gate=rng.random() < 0.7)
    if op == "decode":
        H, G, P, N = _heads(rng)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    state=rng.choice(["f32", "f32", "bf16"]), H=H, G=G, P=P, N=N,
                    batch=_spread(rng, 1, 256), gate=rng.random() < 0.7)
    return dict(op=op, requests=_spread(rng, 1, 4096), most_new=_spread(rng, 1, 128),
                most_ctx=_spread(rng, 1, 16384), page=rng.choice([16, 32, 64, 128]),
                pad=_spread(rng, 1, 1000) - 1)


def _lengths(case):
    """Lengths of the sequences of a prefill case: they add up to its tokens; the larger `spread`,
    the further they are from one another, down to sequences of no token."""
    n, T = case["seqs"], case["tokens"]
    rng = random.Random(n * 1000003 + T)
    share = [1.0 + case["spread"] * (2.0 * rng.random() - 1.0) for _ in range(n)]
    cut = [0] + [int(round(T * sum(share[:i + 1]) / sum(share))) for i in range(n)]
    cut[n] = T
    return [cut[i + 1] - cut[i] for i in range(n)]


def _counts(case):
    """(ctx, new) of the requests of a tables case; every 16th request has nothing to come."""
    n = case["requests"]
    rng = random.Random(n * 1000003 + case["most_new"])
    new = [0 if i % 16 == 15 else rng.randint(1, case["most_new"]) for i in range(n)]
    ctx = [rng.randint(0, case["most_ctx"]) for _ in range(n)]
    return ctx, new


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# ----------------------------------------------------------------------------------- prepare
def prepare(case, seed):
    if case["op"] == "tables":
        return _prepare_tables(case, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    Cc, t = H * P + 2 * G * N, _dtype(case["dtype"])
    lens = _lengths(case) if case["op"] == "prefill" else [1] * case["batch"]
    T = sum(lens)
    s = dict(op=case["op"], H=H, G=G, P=P, N=N)
    s["x"] = normal(T, Cc, dtype=t)
    s["dt"] = normal(T, H, std=0.5)
    s["z"] = normal(T, H, P, dtype=t) if case["gate"] else None
    s["conv_w"] = normal(Cc, CONV, std=0.5, dtype=t)
    s["conv_b"] = normal(Cc, std=0.1, dtype=t)
    # a step of 1e-3 to 1e-1 and decay rates of 1 to 16, even over their logarithm and value
    step = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["a_log"] = torch.log(uniform(H, lo=1.0, hi=16.0))
    s["D"] = 1.0 + normal(H, std=0.1)
    if case["op"] == "decode":
        slots = T + 3
        s["slot"] = torch.randperm(slots, generator=g, device="cuda")[:T].to(torch.int32)
        s["S"] = normal(slots, H, P, N, std=0.1, dtype=_dtype(case["state"]))
        s["conv"] = normal(slots, CONV - 1, Cc, dtype=t)
    else:
        n = len(lens)
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["S0"] = normal(n, H, P, N, std=0.1) if case["init"] else None
        s["conv0"] = normal(n, CONV - 1, Cc, dtype=t) if case["init"] else None
        s["plan"] = _plan(lens)
    return s


def _plan(lens):
    """Index arrays of the plain form: the sequence and the extended row of every token, the
    tokens of every chunk (chunks restart with each sequence), and each chunk's sequence."""
    n_of, ext, rows, seq, first = [], [], [], [], 0
    for n, L in enumerate(lens):
        n_of += [n] * L
        ext += range(first + 3 * (n + 1), first + 3 * (n + 1) + L)
        for c in range(0, L, CHUNK):
            rows.append([first + c + j if c + j < L else -1 for j in range(CHUNK)])
            seq.append(n)
        first += L
    dev = dict(dtype=torch.int64, device="cuda")
    return dict(ext=torch.tensor(ext, **dev), rows=torch.tensor(rows, **dev).view(-1, CHUNK),
                seq=torch.tensor(seq, **dev), lens=torch.tensor(lens, **dev))


def _prepare_tables(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _counts(case)
    n, page = case["requests"], case["page"]
    held = [-(-c // page) for c in ctx]
    need = [-(-(c + v) // page) for c, v in zip(ctx, new)]
    width = max(need) + 1
    slots, pages = n + 5, sum(need) + 64
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    slot = torch.randperm(slots, generator=g, device="cuda")[:n].to(torch.int32)
    # the table as the earlier steps left it: the pages held so far, -1 behind them
    t_held = torch.tensor(held, dtype=torch.int64, device="cuda")
    first = torch.cumsum(t_held, 0) - t_held
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col[None, :]).clamp(max=pages - 1)
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    table[slot.long()] = torch.where(col[None, :] < t_held[:, None], perm[at],
                                     torch.full_like(at, -1, dtype=torch.int32))
    total = sum(new)
    return dict(op="tables", page=page, rows=total + case["pad"],
                ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                new=torch.tensor(new, dtype=torch.int32, device="cuda"), slot=slot,
                table=table, free=perm[sum(held):].contiguous(),
                head=torch.full((1,), seed % 7, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------------------------- run
def run(s):
    if s["op"] == "prefill":
        return _own_prefill(s) if own else _plain_prefill(s)
    if s["op"] == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    return _own_tables(s) if own else _plain_tables(s)


def _own_prefill(s):
    import gated_deltanet_layer_02_b200 as gdn
    return gdn.ssm_prefill(s["x"], s["dt"], s["a_log"], s["cu"], conv_w=s["conv_w"],
                           conv_b=s["conv_b"], dt_bias=s["dt_bias"], D=s["D"], z=s["z"],
                           S0=s["S0"], conv0=s["conv0"], dims=gdn.SsmDims(s["H"], s["G"], s["P"], s["N"]))


def _own_decode(s):
    import gated_deltanet_layer_02_b200 as gdn
    out = gdn.ssm_decode_step(s["x"], s["dt"], s["a_log"], s["conv"], s["S"], s["conv_w"],
                              conv_b=s["conv_b"], dt_bias=s["dt_bias"], D=s["D"], z=s["z"],
                              slot_idx=s["slot"], dims=gdn.SsmDims(s["H"], s["G"], s["P"], s["N"]))
    return out, s["S"], s["conv"]


def _own_tables(s):
    import gated_deltanet_layer_02_b200 as gdn
    t = gdn.batch_tables(s["ctx"], s["new"], s["slot"], s["table"], s["free"], s["head"],
                         page_size=s["page"], num_rows=s["rows"])
    return t.cu_seqlens, t.positions, t.slot_map, t.free_head, s["table"]


# -------------------------------------------------------------------------------- plain forms
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _gates(s):
    """(delta, log of the decay) [T, H] in fp32."""
    raw = s["dt"] + s["dt_bias"]
    delta = torch.clamp(raw, min=0.0) + torch.log1p(torch.exp(-torch.abs(raw)))
    return delta, -torch.exp(s["a_log"]) * delta


def _plain_prefill(s):
    H, G, P, N, plan = s["H"], s["G"], s["P"], s["N"], s["plan"]
    x, w = s["x"], s["conv_w"].float()
    T, Cc, n = x.shape[0], x.shape[1], plan["lens"].numel()
    # rows of every sequence behind its three rows of history
    ext = torch.zeros(T + 3 * n, Cc, dtype=torch.float32, device=x.device)
    ext[plan["ext"]] = x.float()
    start = s["cu"][:-1].long() + 3 * torch.arange(n, device=x.device)
    hist = start[:, None] + torch.arange(3, device=x.device)
    if s["conv0"] is not None:
        ext[hist.reshape(-1)] = s["conv0"].float().reshape(-1, Cc)
    u = ext[plan["ext"] - 3] * w[:, 0] + ext[plan["ext"] - 2] * w[:, 1] \
        + ext[plan["ext"] - 1] * w[:, 2] + ext[plan["ext"]] * w[:, 3] + s["conv_b"].float()
    conv_n = ext[(hist + plan["lens"][:, None]).reshape(-1)].reshape(n, 3, Cc).to(x.dtype)
    del ext
    u = _silu(u)
    delta, la = _gates(s)
    # chunks [c, CHUNK, ...]; what lies behind a sequence's end has delta = 0 and no decay
    rows, keep = plan["rows"].clamp(min=0), plan["rows"] >= 0
    u, delta = u[rows], delta[rows] * keep[..., None]
    cum = torch.cumsum(la[rows] * keep[..., None], 1)                       # [c, i, H]
    xc = u[..., :H * P].unflatten(-1, (H, P))
    Bc = u[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    Cn = u[..., H * P + G * N:].unflatten(-1, (G, N))
    del u
    c = rows.shape[0]
    xd = xc * delta[..., None]
    # the state that each chunk adds, and the state that enters it
    last = cum[:, -1]                                                        # [c, H]
    wx = xd * torch.exp(last[:, None] - cum)[..., None]
    add = torch.einsum("cighp,cign->cghpn", wx.unflatten(2, (G, H // G)), Bc).reshape(c, H, P * N)
    del wx
    before = torch.cumsum(last.double(), 0) - last.double()                  # log decay before c
    seq = plan["seq"]
    first = torch.full((n,), c, device=x.device).scatter_reduce(
        0, seq, torch.arange(c, device=x.device), "amin")
    past = (seq[:, None] == seq[None, :]) & (torch.arange(c, device=x.device)[:, None] >
                                             torch.arange(c, device=x.device)[None, :])
    mix = torch.where(past[None], torch.exp(torch.clamp(
        before.T[:, :, None] - (before + last.double()).T[:, None, :], max=0.0)), 0.0).float()
    enter = (mix @ add.transpose(0, 1)).transpose(0, 1)                      # [c, H, P N]
    del mix
    if s["S0"] is not None:
        since = torch.exp(before - before[first[seq].clamp(max=c - 1)]).float()
        enter = enter + since[..., None] * s["S0"].reshape(n, H, P * N)[seq]
    # the state behind each sequence: that of its last chunk, or the one it began with
    end = torch.exp(last)[..., None] * enter + add
    del add
    SN = torch.zeros(n, H, P * N, device=x.device) if s["S0"] is None else \
        s["S0"].reshape(n, H, P * N).clone()
    is_last = torch.ones(c, dtype=torch.bool, device=x.device)
    is_last[:-1] = seq[1:] != seq[:-1]
    SN[seq[is_last]] = end[is_last]
    del end
    # outputs: what enters, what the chunk itself adds, and the direct term
    y = torch.einsum("cign,cghpn->cighp", Cn, enter.view(c, G, H // G, P, N)).reshape(
        c, CHUNK, H, P) * torch.exp(cum)[..., None]
    del enter
    cb = torch.einsum("cign,cjgn->cgij", Cn, Bc)
    low = torch.tril(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device))
    ct = cum.transpose(1, 2)
    m = torch.exp(torch.where(low, ct[:, :, :, None] - ct[:, :, None, :], -math.inf))
    m = m.unflatten(1, (G, H // G)) * cb[:, :, None]
    y = y + torch.einsum("cghij,cjghp->cighp", m, xd.unflatten(2, (G, H // G))).reshape(
        c, CHUNK, H, P)
    del m
    y = y + s["D"][:, None] * xc
    out = torch.empty(T, H, P, device=x.device)
    out[plan["rows"][keep]] = y[keep]
    if s["z"] is not None:
        out = out * _silu(s["z"].float())
    return out.to(x.dtype), SN.view(n, H, P, N), conv_n


def _plain_decode(s):
    H, G, P, N, slot = s["H"], s["G"], s["P"], s["N"], s["slot"].long()
    x, w = s["x"], s["conv_w"].float()
    ext = torch.cat([s["conv"][slot], x[:, None]], 1)                        # [B, 4, Cc]
    u = _silu((ext.float() * w.T).sum(1) + s["conv_b"].float())
    s["conv"][slot] = ext[:, 1:]
    delta, la = _gates(s)
    xh = u[:, :H * P].unflatten(1, (H, P))
    Bh = u[:, H * P:H * P + G * N].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    Ch = u[:, H * P + G * N:].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    S = s["S"][slot].float() * torch.exp(la)[..., None, None] \
        + (xh * delta[..., None])[..., None] * Bh[:, :, None]
    y = (S * Ch[:, :, None]).sum(-1) + s["D"][:, None] * xh
    s["S"][slot] = S.to(s["S"].dtype)
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(x.dtype), s["S"], s["conv"]


def _plain_tables(s):
    page, rows, dev = s["page"], s["rows"], s["new"].device
    ctx, new, slot = s["ctx"].long(), s["new"].long(), s["slot"].long()
    n, width = new.numel(), s["table"].shape[1]
    cu = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    cu[1:] = torch.cumsum(new, 0)
    held, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    take = torch.cumsum(need - held, 0)
    first = s["head"].long() + take - (need - held)        # place of each request's first new page
    col = torch.arange(width, device=dev)
    fresh = (col >= held[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)
    mine = torch.where(fresh, s["free"][at], s["table"][slot])
    s["table"][slot] = mine
    t = torch.arange(rows, device=dev)
    of = (torch.searchsorted(cu, t, right=True) - 1).clamp(0, n - 1)
    inside = t < cu[-1]
    pos = torch.where(inside, ctx[of] + t - cu[of], -1)
    got = mine[of, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    return (cu.to(torch.int32), pos.to(torch.int32), torch.where(inside, got, -1),
            (s["head"] + take[-1:]).to(torch.int32), s["table"])


# -------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "tables":
        ctx, new = _counts(case)
        n, page, rows = case["requests"], case["page"], sum(new) + case["pad"]
        taken = sum(-(-(c + v) // page) - -(-c // page) for c, v in zip(ctx, new))
        # lengths and slots in, cu_seqlens out; each new page in and out; positions and rows out
        return {"bytes": 12 * n + 4 * (n + 1) + 8 * taken + 12 * rows + 8, "flops": 4 * rows}
    H, G, P, N = case["H"], case["G"], case["P"], case["N"]
    Cc, e = H * P + 2 * G * N, 4 if case["dtype"] == "f32" else 2
    T = case["tokens"] if case["op"] == "prefill" else case["batch"]
    n = case["seqs"] if case["op"] == "prefill" else case["batch"]
    per_token = Cc * e + H * 4 + H * P * e * (2 if case["gate"] else 1)
    weights = Cc * (CONV + 1) * e + 3 * H * 4
    e_state = 2 if case["op"] == "decode" and case["state"] == "bf16" else 4
    sides = 2 if case["op"] == "decode" or case["init"] else 1
    states = sides * n * (H * P * N * e_state + 3 * Cc * e)
    # decay, update and read-out of every element of the state, and the convolution
    flops = T * (5 * H * P * N + 12 * Cc + 8 * H * P)
    return {"bytes": T * per_token + weights + states, "flops": flops}


# ------------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(case, s)
    if case["op"] == "decode":
        slot = s["slot"].long()
        d, S, conv = _exact_layer(s, s["x"][:, None], s["dt"][:, None],
                                  None if s["z"] is None else s["z"][:, None],
                                  s["S"][slot].double(), s["conv"][slot].double(),
                                  [1] * slot.numel())
        S_all, conv_all = s["S"].double(), s["conv"].double()
        S_all[slot], conv_all[slot] = S, conv
        return d[:, 0], S_all, conv_all
    lens, T = _lengths(case), case["tokens"]
    if T > 70000 or max(lens) * len(lens) > 400000:
        return None
    n, longest = len(lens), max(lens)
    H, P, N, Cc = s["H"], s["P"], s["N"], s["x"].shape[1]

    def padded(v):
        if v is None:
            return None
        r = torch.zeros(n, longest, *v.shape[1:], dtype=v.dtype, device=v.device)
        at = 0
        for i, L in enumerate(lens):
            r[i, :L] = v[at:at + L]
            at += L
        return r

    S = torch.zeros(n, H, P, N, dtype=torch.float64, device="cuda") if s["S0"] is None \
        else s["S0"].double()
    conv = torch.zeros(n, 3, Cc, dtype=torch.float64, device="cuda") if s["conv0"] is None \
        else s["conv0"].double()
    d, S, conv = _exact_layer(s, padded(s["x"]), padded(s["dt"]), padded(s["z"]), S, conv, lens)
    out = torch.cat([d[i, :L] for i, L in enumerate(lens)], 0)
    return out, S, conv


def _exact_layer(s, x, dt, z, S, hist, lens):
    """The layer token by token in 64 bits; sequences of a padded batch stop at their lengths."""
    H, G, P, N = s["H"], s["G"], s["P"], s["N"]
    n, longest = x.shape[:2]
    left = torch.tensor(lens, device=x.device)
    w, b = s["conv_w"].double(), s["conv_b"].double()
    A, D = -torch.exp(s["a_log"].double()), s["D"].double()
    out = torch.zeros(n, longest, H, P, dtype=torch.float64, device=x.device)
    for t0 in range(0, longest, 1024):
        t1 = min(longest, t0 + 1024)
        rows = torch.cat([hist, x[:, t0:t1].double()], 1)
        a = b.expand(n, t1 - t0, -1).clone()
        for i in range(CONV):
            a = a + rows[:, i:i + t1 - t0] * w[:, i]
        a = a * torch.sigmoid(a)
        step = torch.nn.functional.softplus(dt[:, t0:t1].double() + s["dt_bias"].double(),
                                            threshold=100.0)
        inside = torch.arange(t0, t1, device=x.device)[None, :] < left[:, None]
        step = step * inside[..., None]          # a step of 0 leaves the state as it is
        decay = torch.exp(step * A)
        xh = a[..., :H * P].reshape(n, t1 - t0, H, P, 1)
        per = H // G
        Bt = a[..., H * P:H * P + G * N].reshape(n, t1 - t0, G, 1, N).expand(
            -1, -1, -1, per, -1).reshape(n, t1 - t0, H, N)
        Ct = a[..., H * P + G * N:].reshape(n, t1 - t0, G, 1, N).expand(
            -1, -1, -1, per, -1).reshape(n, t1 - t0, H, N, 1)
        xs = xh * step[..., None, None]
        for t in range(t1 - t0):
            S = torch.addcmul(S * decay[:, t, :, None, None], xs[:, t], Bt[:, t, :, None])
            out[:, t0 + t] = torch.matmul(S, Ct[:, t]).squeeze(-1)
        out[:, t0:t1] += D[:, None] * xh.squeeze(-1)
        # the three rows before each sequence's next token
        gone = (left - t0).clamp(0, t1 - t0)
        at = gone[:, None] + torch.arange(3, device=x.device)
        hist = torch.gather(rows, 1, at[..., None].expand(-1, -1, rows.shape[2]))
    if z is not None:
        out = out * z.double() * torch.sigmoid(z.double())
    return out, S, hist


def _exact_tables(case, s):
    ctx, new = _counts(case)
    page, free = s["page"], s["free"].tolist()
    head, slot, table = int(s["head"]), s["slot"].tolist(), s["table"].tolist()
    cu, pos, where = [0], [], []
    for n, (c, v) in enumerate(zip(ctx, new)):
        row = table[slot[n]]
        for p in range(-(-c // page), -(-(c + v) // page)):
            row[p] = free[head]
            head += 1
        for q in range(c, c + v):
            pos.append(q)
            where.append(row[q // page] * page + q % page)
        cu.append(cu[-1] + v)
    behind = s["rows"] - len(pos)
    dev = s["new"].device
    return (torch.tensor(cu, dtype=torch.int32, device=dev),
            torch.tensor(pos + [-1] * behind, dtype=torch.int32, device=dev),
            torch.tensor(where + [-1] * behind, dtype=torch.int64, device=dev),
            torch.tensor([head], dtype=torch.int32, device=dev),
            torch.tensor(table, dtype=torch.int32, device=dev))
