"""Plain attention of one request in 64 bits with an element-wise error bound that is derived
key by key, for tests that have to see small faults; and inputs whose result counts the keys
that a row sees.

The bound.  Let w_i = exp(s_i) / sum exp(s), o = sum w_i v_i.  If score i is off by at most
ds_i and the weight's rounding by a factor 1 +- e, then

    |o' - o| <= (sum w_i r_i |v_i - o|  +  sum w_i (1 + r_i) (e |v_i| + dv_i)) / (1 - sum w_i r_i)

with r_i = exp(ds_i) - 1 and dv_i the error of value i.  Proof: the kernels sum the weights before
they are rounded, so o' = sum W_i (1 + E_i) (v_i + D_i) / sum W_i with W_i = w_i (1 + R_i), |R_i| <=
r_i, |E_i| <= e, |D_i| <= dv_i.  Then o' - o = sum W_i (v_i - o) / sum W_i + sum W_i (E_i v_i + (1 +
E_i) D_i) / sum W_i; as sum w_i (v_i - o) = 0, the first numerator is sum w_i R_i (v_i - o) (a common
factor of the scores' errors cancels, the rounding of the weights does not), and sum W_i >= 1 - sum
w_i r_i.  A fp16 weight is 2^(s_i - m + 7), m at most the row's largest score, so below 2^-14 it is off
by half a step of 2^-24, 2^-32 of the row's largest weight, instead: e w_i is at least that.  What ds,
e and dv are is stated per kernel in `attention`."""
import numpy as np

H = 2.0 ** -11      # half a step of fp16, relative


def tanh_cap(s, cap):
    return cap * np.tanh(s / cap) if cap else s


def attention(q, K, V, see, pos_q, pos_k, G, cap=0.0, alibi=None, window=0, scale=0.0, operands="fp16", kmax=None,
              vmax=None, vstep=0.0, kstep=0.0):
    """q [t, Hq, D], K, V [Hkv, n, D], see bool [t, n], positions [t], [n] -> (out, bound) [t, Hq, D].

    operands "fp16" (kvq_tree_attn): keys, values and weights are rounded to fp16, H of themselves
    at most, keys and values by kstep and vstep (absolute; one number or [n]) if that is more; a query or bf16 key row
    is exact to 2^-38 of its largest.  Scores: fp32 sums of D products, accumulated by the
    tensor cores: 2^-19 of the sum of the products' sizes.
    operands "fp32" (kvq_decode_attn_scored): a key is code * s + z, its two parts in products of
    their own whose factors carry 22 bits (hi and lo fp16), summed in fp32: 2^-19 of the parts'
    sizes, which are at most 2 kmax and kmax per channel (kmax: largest |key| of a channel, [Hkv, D];
    max - min <= 2 kmax), and the same for values with vmax ([Hkv, D]).  Weights: 2^-20.
    Both: the exponent's argument in fp32 and its approximation, 2^-20 of |s - max| + 2^-20; the
    cap 2^-20 of itself up to 64, 2^-18 of the score above; the bias 2^-21 of itself."""
    t, Hq, D = q.shape
    scale = scale or D ** -0.5
    out, bound = np.zeros((t, Hq, D)), np.zeros((t, Hq, D))
    dist = pos_q[:, None] - pos_k[None]
    if window:
        see = see & (dist < window)
    fp16 = operands == "fp16"
    e = H if fp16 else 2.0 ** -20
    for h in range(Hq):
        for r in range(t):
            on = np.flatnonzero(see[r])
            if not len(on):
                continue
            k, v = K[h // G][on], V[h // G][on]
            aq, ak = np.abs(q[r, h]), np.abs(k)
            s = (k @ q[r, h]) * scale
            if fp16:
                ds = (np.maximum(H * ak, kstep) + 2.0 ** -19 * ak) @ aq + 2.0 ** -38 * (aq.max() * ak.sum(1) + aq.sum() * ak.max(1))
                dv = np.maximum(H * np.abs(v), vstep if np.ndim(vstep) == 0 else vstep[on][:, None])
            else:
                ds = np.full(len(on), 2.0 ** -19 * 3 * (aq @ kmax[h // G]))
                dv = np.full(v.shape, 2.0 ** -19 * 3) * vmax[h // G]
            ds = abs(scale) * ds
            if cap:
                s = tanh_cap(s, cap)
                ds = ds + (2.0 ** -20 * cap if cap <= 64 else 2.0 ** -18 * np.abs(s))
            if alibi is not None:
                bias = alibi[h] * dist[r][on]
                s = s - bias
                ds = ds + 2.0 ** -21 * np.abs(bias)
            ds = ds + 2.0 ** -20 * (s.max() - s) + 2.0 ** -20 + 2.0 ** -22 * np.abs(s)
            w = np.exp(s - s.max())
            w /= w.sum()
            o = w @ v
            f = w * (np.exp(ds) - 1)
            left = max(1 - f.sum(), 0.1)
            out[r, h] = o
            ew = np.maximum(e * (w + f), 2.0 ** -32 * (w + f).max()) if fp16 else e * (w + f)
            bound[r, h] = (f @ np.abs(v - o) + ew @ np.abs(v) + (w + f + ew) @ dv) / left + 2.0 ** -22 * np.abs(o)
    return out, bound


def counting_values(n, D, bits):
    """Values [n, D] that name their token: token i has 2^bits - 1 in channel i % D, else 0 (a
    quantizer with scale 1 or 0 and zero 0 keeps them).  With equal keys a row's output in channel
    c, times the number of keys it sees, over 2^bits - 1, is the number of them with i % D == c."""
    v = np.zeros((n, D))
    v[np.arange(n), np.arange(n) % D] = 2 ** bits - 1
    return v


def counts(see_tokens, D):
    """Number of seen tokens per channel, [D], from their indices."""
    return np.bincount(np.asarray(see_tokens, np.int64) % D, minlength=D).astype(np.float64)
