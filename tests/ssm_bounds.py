"""Error bounds of a bf16 prompt of at most one chunk (128 tokens) from the fp16 operands that the
chunked form has, derived element by element.

An operand v is kept as fp16(v 2^s), s an exponent shared by what is scaled together.  fp16 is off
by at most 2^-11 of a value (half a step), and by at most 2^-25 of the scaled one however small it
is.  With the largest magnitudes X_j of the 64 channels of x of token j, B_j, C_i of its rows of B
and C, and S of the 64 rows of a state:
  C     2^4  > max >= 2^3 :  2^-11 |C|,  2^-28 C_i
  B     2^14 > max >= 2^13:  2^-11 |B|,  2^-38 B_j
  C.B   kept 2^10 smaller than the product of the two:  2^-11 |C.B|,  2^-25-16+10 C_i B_j
  P     C.B times a weight that is 1 for the token with the largest w X_j B_j:  2^-11 |P|, and
        2^-25 in units that make its product with x 2^-31 |x_jp| / 2^(exponent of X_j) C_i max(w X B):
        2^-30 |x_jp| / X_j C_i max_j(w_ij X_j B_j)
  x     2^14 > max >= 2^13:  2^-11 |x|,  2^-38 X_j
  S     2^15 > max >= 2^14:  2^-11 |S|,  2^-39 S
So a term of P x is rounded five times, one of C S twice, D x once.  The state's factors have two
parts each, 2^-22 of the value; the second part too ends at 2^-25 of the scaled value:
  B     2^-38 B_j;   w x   2^14 > max >= 2^12 by the factors' exponents:  2^-36 |B_jn| / B_j max(w X B)
fp32 arithmetic around it (conv, silu, gates, sums): 2^-13 for outputs and 2^-14 for states, as in
ssm_util.  Where the conv is one tap of weight 1, so that nothing cancels, the values are below 8 and
the decays slow, that is less (TIGHT_*).  A silu is off by 2^-20.5 (exp2 2 units of 2^-23 and up to
2^-21 from its argument, reciprocal, sum and product one each), a weight by 2^-20, two parts leave
3 2^-22 (each factor, and the product of the two second parts).  Products are summed 16 at a time; each
addend counts as off by 2^-23 of the largest.  A state of at most 5 tokens is 3 such sums of 6 addends:
2 2^-20.5 + 2^-20 + 3 2^-22 + 18 2^-23 < 2^-17.  An output has a third factor, and C.B and C S are 8 sums
of 17: 3 2^-20.5 + 2^-20 + (136 + 6) 2^-23 < 2^-15.
"""
import numpy as np

import ssm_util as U

FIVE = 5.02 * 2.0 ** -11   # (1 + 2^-11)^5 - 1
HALF_BF16 = 2.0 ** -8
TIGHT_OUT, TIGHT_STATE = 2.0 ** -15, 2.0 ** -17


def chunk_bounds(i, H, G, P, N, out_rel=2.0 ** -13, state_rel=2.0 ** -14):
    """(out, SN, out bound, SN bound) in fp64 of sequences of at most 128 tokens, without history."""
    out, SN, _, s_out, s_SN = U.layer(i, H, G, P, N)
    b_out, b_SN = (FIVE + out_rel) * s_out, state_rel * s_SN
    x, w, cu, per = U.f64(i["x"]), U.f64(i["conv_w"]), i["cu"].numpy(), H // G
    delta = U.softplus(U.f64(i["dt"]) + (0.0 if i["dt_bias"] is None else U.f64(i["dt_bias"])))
    lam = -np.exp(U.f64(i["a_log"])) * delta
    D = np.zeros(H) if i["D"] is None else np.abs(U.f64(i["D"]))
    g = 1.0 if i["z"] is None else np.abs(U.silu(U.f64(i["z"])))
    extra = np.zeros_like(out)
    for n in range(len(cu) - 1):
        s, e = int(cu[n]), int(cu[n + 1])
        assert e - s <= 128 and i["conv0"] is None
        rows = np.concatenate([np.zeros((3, x.shape[1])), x[s:e]])
        a = sum(rows[j:j + e - s] * w[:, j] for j in range(4))
        u = np.abs(U.silu(a + (0.0 if i["conv_b"] is None else U.f64(i["conv_b"]))))
        for h in range(H):
            k, cB = h // per, H * P + (h // per) * N
            Bu, Cu = u[:, cB:cB + N], u[:, cB + G * N:cB + G * N + N]
            Bm, Cm = Bu.max(1, initial=0.0), Cu.max(1, initial=0.0)
            cum = np.cumsum(lam[s:e, h])
            low = np.tril(np.ones((e - s, e - s)))
            W = np.exp(np.minimum(cum[:, None] - cum[None, :], 0.0)) * low * delta[s:e, h]
            WL = np.exp(cum[-1:] - cum) * delta[s:e, h]
            CB = Cu @ Bu.T
            S0 = np.zeros((P, N)) if i["S0"] is None else np.abs(U.f64(i["S0"])[n, h])
            dec = np.exp(cum)
            for p0 in range(0, P, 64):
                xs = u[:, h * P + p0:h * P + p0 + 64]
                Xm, S = xs.max(1, initial=0.0), S0[p0:p0 + 64]
                safe = np.where(Xm > 0, Xm, 1.0)
                top = (W * (Xm * Bm)).max(1, initial=0.0)
                v = 2.0 ** -28 * Cm[:, None] * (W @ (xs * Bu.sum(1, keepdims=True)) +
                                                dec[:, None] * S.sum(1))
                v += 2.0 ** -38 * Cu.sum(1, keepdims=True) * (W @ (xs * Bm[:, None]))
                v += 2.0 ** -31 * Cm[:, None] * (W @ (xs * Bm[:, None]))
                v += 2.0 ** -30 * (Cm * top)[:, None] * (low @ (xs / safe[:, None]))
                v += 2.0 ** -38 * (((W * CB) @ Xm) + D[h] * Xm)[:, None]
                v += 2.0 ** -39 * (dec * Cu.sum(1))[:, None] * S.max(initial=0.0)
                extra[s:e, h, p0:p0 + 64] = v
                topL = (WL * Xm * Bm).max(initial=0.0)
                frac = (Bu / np.where(Bm > 0, Bm, 1.0)[:, None]).sum(0)
                b_SN[n, h, p0:p0 + 64] += 2.0 ** -38 * ((WL * Bm) @ xs)[:, None] + \
                    2.0 ** -36 * topL * frac[None, :]
    return out, SN, b_out + extra * g + HALF_BF16 * np.abs(out) + 2.0 ** -100, b_SN + 2.0 ** -100


def worst(got, ref, bound):
    """Largest error in units of the bound."""
    g = U.f64(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g))
    return float(np.max(np.abs(g - ref) / bound)) if ref.size else 0.0
