"""fp64 definitions of the operators beside the gated delta rule (include/gdn.h), token by
token in numpy, with the error bounds the GPU tests hold the kernels to.

TEST INFRASTRUCTURE ONLY, like the rest of this package; no code is shared with csrc/.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24    # half a step of fp32


def gates(x, a, b, A_log, dt_bias):
    """(z, E, g, alpha, s, beta, u) of the gated linear recurrence, broadcast over channels last."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    z = a + np.asarray(dt_bias, np.float64)
    E = np.exp(np.asarray(A_log, np.float64))
    g = -E * np.logaddexp(0.0, z)
    s = np.sqrt(-np.expm1(2.0 * g))
    beta = np.where(b >= 0, 1.0 / (1.0 + np.exp(-np.abs(b))), np.exp(-np.abs(b)) / (1.0 + np.exp(-np.abs(b))))
    return z, E, g, np.exp(g), s, beta, s * beta * x


def recurrence(x, a, b, A_log, dt_bias, starts, initial_state=None, dout=None, dfinal=None):
    """Over flattened tokens [Ntok, D] with sequences starts[n] .. starts[n+1]. Returns a dict with
    out and final, with dout also the gradients, and for each a bound ``*_err`` on what fp32
    arithmetic in any order of the scan may add (the rounding of the result to the activation type not
    included).

    Bounds. kappa is the relative error of alpha, u and of one step's products in fp32: the rounding of
    z and of the exponent's argument move softplus by up to 2 |z| U32 relative, the polynomials,
    exponentials, reciprocals and roots by a few U32 each, 24 in all. It is carried through the
    recurrences exactly as the values are. Below fp32's normal range the kernels' exponentials count as 0:
    t = e^-|z| is off by at most 2^-126 then, so -g by E 2^-126 and w = -expm1(2g) by 2 E 2^-126; and a w below
    2^-126 counts as 0 itself. sqrt(p + q) - sqrt(p) <= sqrt(q), so s is off by at most fs = (sqrt(2E) + 1) 2^-63
    there, and beta (whose e^-b may overflow, or whose value flush) by fb = 2^-126. In da the factor E sigmoid(z)
    alpha^2 / s is taken as 0 where s is; its value is at most E e^z / sqrt(2 E e^z (1 - E e^z)) there, which is
    below fs / 2, and times |g| / (E sigmoid(z)) <= 1 + fs it enters dA_log.
    """
    z, E, g, alpha, s, beta, u = gates(x, a, b, A_log, dt_bias)
    n_tok, D = z.shape
    N = len(starts) - 1
    kappa = (2.0 * np.abs(z).max(initial=0.0) + 24.0) * U32
    fs, fb = (np.sqrt(2.0 * E) + 1.0) * 2.0 ** -63, 2.0 ** -126
    floor = (beta * fs + s * fb) * np.abs(np.asarray(x, np.float64))
    h0 = np.zeros((N, D)) if initial_state is None else np.asarray(initial_state, np.float64)
    h, eh = np.zeros((n_tok, D)), np.zeros((n_tok, D))
    before, ebefore = np.zeros((n_tok, D)), np.zeros((n_tok, D))
    final, efinal = h0.copy(), np.zeros((N, D))
    for n in range(N):
        c, ec = h0[n], np.zeros(D)
        for t in range(starts[n], starts[n + 1]):
            before[t], ebefore[t] = c, ec
            ec = alpha[t] * ec + kappa * (alpha[t] * np.abs(c) + np.abs(u[t])) + floor[t]
            c = alpha[t] * c + u[t]
            h[t], eh[t] = c, ec
        final[n], efinal[n] = c, ec
    r = {"out": h, "out_err": eh, "final": final, "final_err": efinal}
    if dout is None:
        return r
    dout = np.asarray(dout, np.float64)
    df = np.zeros((N, D)) if dfinal is None else np.asarray(dfinal, np.float64)
    delta, ed = np.zeros((n_tok, D)), np.zeros((n_tok, D))
    dstate, estate = df.copy(), np.zeros((N, D))
    for n in range(N):
        c, ec = df[n], np.zeros(D)
        for t in reversed(range(starts[n], starts[n + 1])):
            delta[t] = dout[t] + c
            ed[t] = ec + 2 * U32 * (np.abs(dout[t]) + np.abs(c))
            c, ec = alpha[t] * delta[t], alpha[t] * ed[t] + kappa * alpha[t] * np.abs(delta[t])
        dstate[n], estate[n] = c, ec
    x = np.asarray(x, np.float64)
    sig = np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
    with np.errstate(divide="ignore", invalid="ignore"):
        inv_s = np.where(s > 0, alpha * alpha / s, 0.0)
    m1, m2 = alpha * before, beta * x * inv_s
    dg, edg = delta * (m1 - m2), ed * np.abs(m1 - m2) + np.abs(delta) * (alpha * ebefore + kappa * (np.abs(m1) + np.abs(m2)))
    r["dx"], r["dx_err"] = delta * s * beta, (ed + kappa * np.abs(delta)) * s * beta + np.abs(delta) * (beta * fs + s * fb)
    r["db"] = delta * s * beta * (1.0 - beta) * x
    # 1 - beta of a beta near 1 keeps an absolute error of a few U32
    r["db_err"] = (ed + kappa * np.abs(delta)) * s * beta * (1.0 - beta + 4 * U32) * np.abs(x) + \
        np.abs(delta) * (s * beta * 4 * U32 * np.abs(x) + floor)
    r["da"], r["da_err"] = -dg * E * sig, E * sig * (edg + kappa * np.abs(dg)) + \
        np.abs(delta) * (floor + E * fb * (np.abs(m1) + np.abs(m2)))
    r["dstate"], r["dstate_err"] = dstate, estate
    # sums over tokens in fp32: at most one rounding per addend, of a partial sum no larger than sum |addend|
    add = (n_tok + 8) * U32
    for name, v, ev in (("dA_log", dg * g, (edg + kappa * np.abs(dg)) * np.abs(g) + 2 * np.abs(delta) * floor), ("ddt_bias", r["da"], r["da_err"])):
        r[name] = v.sum(0)
        r[name + "_err"] = ev.sum(0) + add * np.abs(v).sum(0)
    return r


def rotary(x, positions, freq, rot, layout, inverse=False, scale=1.0):
    """x [..., T, H, d] with integer positions [..., T] and fp64 radians per position freq [rot/2]."""
    y = np.array(x, np.float64)
    angle = np.asarray(positions, np.int64)[..., None].astype(np.float64) * np.asarray(freq, np.float64)
    c, s = np.cos(angle)[..., None, :] * scale, np.sin(angle)[..., None, :] * scale
    s = -s if inverse else s
    half = rot // 2
    i1 = np.arange(half) if layout == "half" else 2 * np.arange(half)
    i2 = i1 + half if layout == "half" else i1 + 1
    x1, x2 = y[..., i1].copy(), y[..., i2].copy()
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def frequencies(rot, theta=10000.0, scaling="plain", factor=1.0, low=1.0, high=4.0, original=8192.0):
    """fp64 radians per position of every pair (gdn_rotary_scaling in include/gdn.h)."""
    f = float(theta) ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        keep = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        return keep * f + (1.0 - keep) * f / factor
    return f


def group_norm(x, weight, bias, groups, act, eps, dout=None):
    """x [N, L, C]; a dict with out, mean, rstd and, with dout, the gradients; ``*_err`` as above.

    Bounds. mean and the sum of squares of fp32 terms, added in any order: relative to the mean absolute
    (squared) term at most (count + 8) U32, and in practice a tree's (log2 count); k below counts a tree
    over 32 lanes and serial runs of at most ``run`` addends per lane.
    """
    x = np.asarray(x, np.float64)
    N, L, C = x.shape
    cg = C // groups
    y = x.reshape(N, L, groups, cg)
    mean = y.mean((1, 3), keepdims=True)
    var = ((y - mean) ** 2).mean((1, 3), keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    xh = (y - mean) * rstd
    w = np.ones(C) if weight is None else np.asarray(weight, np.float64)
    bb = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    w4, b4 = w.reshape(1, 1, groups, cg), bb.reshape(1, 1, groups, cg)
    z = xh * w4 + b4
    k = (min(L * cg, 4096) + 32) * U32
    mabs = np.abs(y).mean((1, 3), keepdims=True)
    em = k * mabs                                     # mean
    # the centred values move by em and by a rounding of x - mean; the variance by k and the centre's shift squared
    ex = (em + 2 * U32 * (np.abs(y) + np.abs(mean))) * rstd
    exh = ex + np.abs(xh) * (k + 0.5 * (2 * em * rstd * k + (em * rstd) ** 2) + 4 * U32)
    ez = np.abs(w4) * exh + 4 * U32 * (np.abs(xh * w4) + np.abs(b4))
    sg = 1.0 / (1.0 + np.exp(-np.clip(z, -700, 700))) if act == "silu" else np.ones_like(z)
    out = z * sg
    # |d silu| <= 1.1; the sigmoid's own error: the exponent's argument (|z| U32) and a few U32
    eo = 1.1 * ez + np.abs(out) * (np.abs(z) + 8) * 2 * U32 if act == "silu" else ez
    shape = (N, L, C)
    r = {"out": out.reshape(shape), "out_err": eo.reshape(shape), "mean": mean.reshape(N, groups),
         "mean_err": em.reshape(N, groups), "rstd": rstd.reshape(N, groups),
         "rstd_err": (rstd * (k + (em * rstd) ** 2 + 4 * U32)).reshape(N, groups)}
    if dout is None:
        return r
    dy = np.asarray(dout, np.float64).reshape(y.shape)
    da = sg * (1.0 + z * (1.0 - sg)) if act == "silu" else np.ones_like(z)
    # |act''| <= 0.5 for silu
    eda = 0.5 * ez + (np.abs(z) + 8) * 4 * U32 if act == "silu" else np.zeros_like(z)
    dz, edz = dy * da, np.abs(dy) * (eda + 4 * U32)
    t, et = dz * w4, np.abs(w4) * (edz + 4 * U32 * np.abs(dz))
    m1, m2 = t.mean((1, 3), keepdims=True), (t * xh).mean((1, 3), keepdims=True)
    em1 = et.mean((1, 3), keepdims=True) + k * np.abs(t).mean((1, 3), keepdims=True)
    em2 = (et * np.abs(xh) + np.abs(t) * exh).mean((1, 3), keepdims=True) + k * np.abs(t * xh).mean((1, 3), keepdims=True)
    inner = t - m1 - xh * m2
    r["dx"] = (rstd * inner).reshape(shape)
    r["dx_err"] = (rstd * (et + em1 + np.abs(xh) * em2 + exh * np.abs(m2) + 8 * U32 * (np.abs(t) + np.abs(m1) + np.abs(xh * m2))) +
                   np.abs(rstd * inner) * (k + (em * rstd) ** 2 + 4 * U32)).reshape(shape)
    add = (min(N * L, 8192) + 32) * U32
    for name, v, ev in (("dweight", dz * xh, edz * np.abs(xh) + np.abs(dz) * exh), ("dbias", dz, edz)):
        r[name] = v.sum((0, 1)).reshape(C)
        r[name + "_err"] = (ev.sum((0, 1)) + add * np.abs(v).sum((0, 1))).reshape(C)
    return r


# half a step of the activation types, relative, and half of their smallest step
HALF_STEP = {"fp32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25)}


def bound(ref, err, dtype):
    """The tolerance of a result computed within ``err`` in fp32 and rounded once to dtype."""
    rel, least = HALF_STEP[dtype]
    return np.abs(ref) * rel + err * (1.0 + rel) + least
