"""A bar on the norm of a paged attention output's error, tight enough that a mask that is off by one position or a scale off
by a tenth does not pass (the bar of every element in tests/test_gpu_paged.py adds up worst cases, which for 16-bit types is wider).

The error of out = sum_p w_p V_p is propagated to first order, from roundings that are independent of one another and
at most half a step r of the value each; the mean square of one is taken as r^2 / 3 (evenly spread over the step: less, as
the value is between 1 and 2 times the one whose half step is r):
  * the output:  r = eps / 2,  (r out_j)^2 / 3;
  * a weight, r_w:  sum_p (w_p (V_pj - out_j))^2 r_w^2 / 3  (a common factor of all weights drops out);
  * q'_d = q_d s_d, r_q, the same for every position:  out_j moves by scale q_d Cov_w(K_d, V_j):
    sum_d (scale q_d Cov_dj)^2 r_q^2 / 3.
Errors that need not be independent are added as they are:
  * codes that enter a product as subnormals lose up to 2^-14 of it (6e-5): of sum_p w_p code_pj s_j for V; for K a score
    is off by 2^-14 scale sum_d |q_d s_d| code_pd, and out_j by sum_p w_p |V_pj - out_j| times that;
  * 2^-13 of sum_p w_p |V_pj - out_j| for the exponentials (a cubic of relative error 7.5e-5 among them, 2^-13.7) and what is
    rounded in fp32; 2^-20 of sum_p w_p code_pj s_j + |z_j s_j| for the sums.
The bar is 1.5 times the root of the sum of the mean squares over all outputs, and the norm of the rest.

Which roundings there are, by type, new rows and sums, is in `roundings`."""
import math

import numpy as np
import torch

import oracle.paged as paged

TD = {"f16": torch.float16, "bf16": torch.bfloat16}


def roundings(c, G, dtype):
    """(r_q, r_w, K's codes subnormal, V's codes subnormal) of the kernel that takes the call."""
    rows, sums = c.max_q * G, c.w0 is not None
    if rows <= (8 if sums else 16 if dtype == "f16" else 32):  # few rows to a K/V head
        if dtype == "bf16" and not sums:
            return 2.0 ** -11, 2.0 ** -11, True, True
        return 2.0 ** -20, 2.0 ** -20, False, True
    return (2.0 ** -20 if sums else 2.0 ** -11), 2.0 ** -11, False, False


def bar(c, q64, parts, out, dtype, scale):
    """(norm of the reference, bar on the norm of the error)."""
    H, D = c.H, c.D
    G = q64.shape[1] // H
    r_q, r_w, sub_k, sub_v = roundings(c, G, dtype)
    ch = lambda cal: [a.astype(np.float64).reshape(H, D).repeat(G, axis=0) for a in (cal[1][cal[0]], cal[2][cal[0]])]  # noqa: E731
    (sk, zk), (sv, zv) = ch(c.k_cal), ch(c.v_cal)
    square, rest = 0.0, 0.0
    for b, (K, V, _, w) in enumerate(parts):
        for i in range(c.start[b + 1] - c.start[b]):
            for a in range(q64.shape[1]):
                o, wp, q = out[c.start[b] + i, a], w[a, i], q64[c.start[b] + i, a]
                dv = V[:, a] - o
                cov = (K[:, a] * wp[:, None]).T @ dv
                square += (o ** 2).sum() * (torch.finfo(TD[dtype]).eps / 2) ** 2 / 3
                square += ((wp[:, None] * dv) ** 2).sum() * r_w ** 2 / 3
                square += ((scale * q[:, None] * cov) ** 2).sum() * r_q ** 2 / 3
                mag = wp @ np.abs(dv)
                code = wp @ (V[:, a] + zv[a] * sv[a])
                e = 2.0 ** -13 * mag + 2.0 ** -20 * (code + np.abs(zv[a] * sv[a]))
                if sub_v:
                    e = e + 2.0 ** -14 * code
                if sub_k:
                    s = 2.0 ** -14 * scale * (K[:, a] / sk[a] + zk[a]) @ np.abs(q * sk[a])
                    e = e + (wp * s) @ np.abs(dv)
                rest += (e ** 2).sum()
    return math.sqrt((out[:c.start[-1]] ** 2).sum()), 1.5 * math.sqrt(square) + math.sqrt(rest)


def queries(c, G, dtype):
    """Queries of a softmax that is flat enough for a single position's weight to count (the largest is 0.1 to 0.4)."""
    return (c.queries(c.H * G, dtype) * 0.4).to(TD[dtype])


def check_norm(c, q64, got, dtype, reference=None):
    """got [T, Hq, D] against the definition, in norm.  Returns (error, bar) relative to the reference's norm."""
    scale = 1 / math.sqrt(c.D)
    out, _, parts = reference or paged.attention(q64, c.start, c.lens, c.table, c.k0, c.v0, c.k_cal, c.v_cal, c.bits)
    n, t = c.start[-1], bar(c, q64, parts, out, dtype, scale)
    err = math.sqrt(((got[:n] - out[:n]) ** 2).sum())
    assert err <= t[1], f"error {err / t[0]:.3e} of the norm, bar {t[1] / t[0]:.3e}"
    return err / t[0], t[1] / t[0]


# (H, group, D, bits, page, new rows, lengths, dtype, sums): every 16-bit kernel, with and without positions in parts
CASES = [
    (4, 1, 128, 3, 64, [1, 1, 1], [70, 33, 64], "bf16", False),
    (4, 1, 64, 4, 16, [1, 1], [90, 17], "f16", False),
    (2, 2, 128, 4, 16, [1, 2], [80, 60], "bf16", False),
    (2, 4, 64, 3, 32, [1, 3], [50, 70], "f16", False),
    (2, 2, 128, 3, 16, [2, 1], [40, 75], "f16", True),
    (2, 1, 64, 4, 64, [60, 20], [70, 35], "f16", False),
    (2, 1, 128, 3, 16, [60, 20], [70, 35], "bf16", False),
    (1, 2, 128, 4, 32, [40, 30], [60, 30], "f16", False),
    (1, 2, 64, 3, 16, [40, 30], [60, 30], "bf16", False),
    (1, 1, 128, 3, 16, [40, 3], [64, 1100], "f16", False),   # two parts
    (1, 1, 64, 4, 64, [40, 3], [64, 1100], "bf16", False),
    (1, 2, 128, 3, 64, [40, 30], [60, 30], "bf16", True),
    (1, 1, 64, 4, 16, [40, 3], [64, 1100], "f16", True)]
