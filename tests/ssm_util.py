"""fp64 references of the state space layer and of the batch tables, and seeded inputs for them."""
import numpy as np
import torch


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return v / (1.0 + np.exp(-v))


def f64(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def inputs(H, G, P, N, lens, dtype, seed, init=True, gate=True, bias=True, direct=True, std=1.0):
    """CPU tensors of one prefill call (or, with lens all 1, one decode call)."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, k=1.0: k * torch.randn(*s, generator=gen)  # noqa: E731
    T, n, Cc = sum(lens), len(lens), H * P + 2 * G * N
    return dict(
        x=r(T, Cc, k=std).to(dtype), dt=r(T, H, k=0.5), conv_w=r(Cc, 4, k=0.5).to(dtype),
        conv_b=r(Cc, k=0.1).to(dtype) if bias else None,
        dt_bias=r(H) - 2.0 if bias else None,
        a_log=torch.log(1.0 + 15.0 * torch.rand(H, generator=gen)),
        D=1.0 + r(H, k=0.1) if direct else None,
        z=r(T, H, P).to(dtype) if gate else None,
        cu=torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32),
        S0=r(n, H, P, N, k=0.1 * std) if init else None,
        conv0=r(n, 3, Cc, k=std).to(dtype) if init else None)


def layer(i, H, G, P, N, dt_min=0.0, dt_max=np.inf, S0=None):
    """(out, SN, convN, out_scale, SN_scale) in fp64.  The scales are the sums of the absolute
    values of what is added up to form each element, so that the error of a sum whose terms are
    each known to a relative eps is at most eps times them."""
    x, cu = f64(i["x"]), i["cu"].numpy()
    w, b = f64(i["conv_w"]), f64(i["conv_b"])
    T, Cc, n, per = x.shape[0], x.shape[1], len(cu) - 1, H // G
    raw = f64(i["dt"]) + (0.0 if i["dt_bias"] is None else f64(i["dt_bias"]))
    delta = np.clip(softplus(raw), dt_min, dt_max)
    decay = np.exp(-np.exp(f64(i["a_log"])) * delta)
    D = np.zeros(H) if i["D"] is None else f64(i["D"])
    S0 = f64(i["S0"]) if S0 is None else S0
    out, scale = np.zeros((T, H, P)), np.zeros((T, H, P))
    SN, MN, conv = np.zeros((n, H, P, N)), np.zeros((n, H, P, N)), np.zeros((n, 3, Cc))
    for k in range(n):
        s, e = int(cu[k]), int(cu[k + 1])
        rows = np.concatenate([np.zeros((3, Cc)) if i["conv0"] is None else f64(i["conv0"])[k],
                               x[s:e]])
        a = sum(rows[j:j + e - s] * w[:, j] for j in range(4))
        m = sum(np.abs(rows[j:j + e - s] * w[:, j]) for j in range(4))
        if b is not None:
            a, m = a + b, m + np.abs(b)
        u, um = silu(a), np.maximum(np.abs(silu(a)), 2.0 ** -6 * m)  # see the tolerance
        S = np.zeros((H, P, N)) if S0 is None else S0[k].copy()
        M = np.abs(S)
        for t in range(e - s):
            q, qm = u[t], um[t]
            xh, xm = q[:H * P].reshape(H, P), qm[:H * P].reshape(H, P)
            B, Bm = (np.repeat(v[H * P:H * P + G * N].reshape(G, N), per, 0) for v in (q, qm))
            C, Cm = (np.repeat(v[H * P + G * N:].reshape(G, N), per, 0) for v in (q, qm))
            d, al = delta[s + t][:, None, None], decay[s + t][:, None, None]
            S = al * S + d * xh[:, :, None] * B[:, None]
            M = al * M + d * xm[:, :, None] * Bm[:, None]
            out[s + t] = (S * C[:, None]).sum(-1) + D[:, None] * xh
            scale[s + t] = (M * Cm[:, None]).sum(-1) + np.abs(D)[:, None] * xm
        SN[k], MN[k], conv[k] = S, M, rows[e - s:]
    if i["z"] is not None:
        g = silu(f64(i["z"]))
        out, scale = out * g, scale * np.abs(g)
    return out, SN, conv, scale, MN


#: Relative error of the terms of a sum, in units of what they are made of.
#: State: delta x B has two factors in two bf16 parts each.  A part is off by at most half a step,
#: 2^-8 of the value, so two parts leave 2^-16 of each factor, and the product of the two second
#: parts, left out, is another 2^-16: 3 2^-16.  The fp32 arithmetic around it (four conv products,
#: exp and division of the silu, softplus, exp of a sum of up to 128 step sizes, fp32 sums) stays
#: below another 2^-16: 2^-14 in all.
#: Outputs: two more factors (state and C, or decay-weighted scores and x).  fp32 activations keep
#: them in two parts too: 2 2^-14.  bf16 activations round each to 11 bits once, 2^-11: two factors
#: are 2^-10, plus the state's 2^-14 and the scores' 2^-14; then one rounding of the result to bf16,
#: 2^-8 of it.
#: (Factors in two fp16 parts, 11 bits each, leave less: the bounds hold for both.)
#: The silu of a conv sum a = sum of terms with magnitude m is off by at most 1.1 eps m; relative to
#: its value that is unbounded near a zero of the sum, so a factor counts with at least 2^-6 m:
#: 2^-24 4 m (the fp32 sum) over 2^-6 m is 2^-16.
STATE = 2.0 ** -14
OUT_F32 = 2.0 ** -13
OUT_BF16 = 2.0 ** -10 + 2.0 ** -13


def check(got, ref, scale, eps, what, half=0.0):
    g = f64(got)
    assert g.shape == ref.shape, what
    assert np.all(np.isfinite(g)), f"{what}: non-finite values"
    bound = eps * scale + half * np.abs(ref) + 2.0 ** -100
    worst = float(np.max(np.abs(g - ref) / bound)) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def check_layer(got, ref, dtype, what):
    out, SN, conv = got
    r_out, r_SN, r_conv, s_out, s_SN = ref
    bf = dtype == torch.bfloat16
    check(out, r_out, s_out, OUT_BF16 if bf else OUT_F32, what + ": out", 2.0 ** -8 if bf else 0.0)
    if SN is not None:
        check(SN, r_SN, s_SN, STATE, what + ": state")
    if conv is not None:
        np.testing.assert_array_equal(f64(conv), r_conv, err_msg=what + ": conv history")


def tables(ctx, new, slot, table, free, head, page, rows):
    """Plain tables: (cu, positions, slot_map, head, table), lists and an array."""
    table, cu, pos, where = np.array(table), [0], [], []
    for n, (c, v) in enumerate(zip(ctx, new)):
        for p in range(-(-c // page), -(-(c + v) // page)):
            table[slot[n], p] = free[head]
            head += 1
        for q in range(c, c + v):
            pos.append(q)
            where.append(int(table[slot[n], q // page]) * page + q % page)
        cu.append(cu[-1] + v)
    pad = [-1] * (rows - len(pos))
    return cu, pos + pad, where + pad, head, table
