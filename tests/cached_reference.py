"""The compressed source cache in 64 bits: the record format from its
definition, the read over the values that records stand for, its gradient, and
for every result how far FP32 arithmetic may be from it.

The bounds count roundings.  u = 2^-24 is the most one FP32 rounding moves a
value, relative.  A sum over a token's channels is at most K = 80 roundings
deep (up to 32 products and sums in a thread, 5 steps over a warp, 8 warps, the
factors before and after); a sum over tokens is as deep as it has terms.
bf16 results are rounded once, by at most 2^-8 of their value.
"""
import struct

import numpy as np

U = 2.0 ** -24
K = 80
EPS = 2.0 ** -23
GRID = {
    4: np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64),
    8: np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127], np.float64),
}


def offsets(D, bits):
    codes = -(-(D * bits // 8) // 16) * 16
    stat = codes + -(-(-(-D // 32)) // 8) * 8
    return codes, stat, -(-(stat + 8) // 16) * 16


def tag(R, ko, bits):
    return R | ko << 14 | (bits == 8) << 27 | 5 << 28


def group_exponent(top, bits):
    """The smallest k >= -110 with top <= largest * 2^k."""
    k = -110
    while top > GRID[bits][-1] * 2.0 ** k:
        k += 1
    return k


def write_row(x, bits, R, ko):
    """One record's bytes (a bytearray) from float64 channels, and the values it stands for."""
    D = len(x)
    codes_n, stat_at, size = offsets(D, bits)
    rec = bytearray(size)
    vals = np.zeros(D)
    for g in range(-(-D // 32)):
        xs = x[32 * g:32 * g + 32]
        if not np.isfinite(xs).all():
            rec[codes_n + g] = 255
            vals[32 * g:32 * g + 32] = np.nan
            continue
        xs = np.clip(xs, -1.5 * 2.0 ** 127, 1.5 * 2.0 ** 127)
        k = group_exponent(np.abs(xs).max(), bits)
        rec[codes_n + g] = k + 127
        a = np.abs(xs) / 2.0 ** k
        mid = (GRID[bits][1:] + GRID[bits][:-1]) / 2
        lo, hi = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
        code = np.where(lo % 2 == 0, lo, hi)          # they differ on a tie alone
        neg = np.signbit(xs)
        vals[32 * g:32 * g + 32] = np.where(neg, -1, 1) * GRID[bits][code] * 2.0 ** k
        for i, c in enumerate(code):
            j = 32 * g + i
            if bits == 8:
                rec[j] = int(c) | (128 if neg[i] else 0)
            else:
                rec[j // 2] |= (int(c) | (8 if neg[i] else 0)) << 4 * (j % 2)
    with np.errstate(over="ignore"):
        ms = np.float32((vals[ko:ko + R] ** 2).sum() / R)
    rec[stat_at:stat_at + 4] = struct.pack("<f", ms)
    rec[stat_at + 4:stat_at + 8] = struct.pack("<I", tag(R, ko, bits))
    return rec, vals


def read(v, q, scale, ko, w=None, dy=None, eps=EPS):
    """v [S, N, D], q [R], w [D], dy [N, D] in float64.  Returns {name: (value, bound)}."""
    S, N, D = v.shape
    R = len(q)
    t = v[..., ko:ko + R]
    r = 1 / np.sqrt((t ** 2).mean(-1) + eps)
    z = scale * r * (t @ q)
    e_z = abs(scale) * r * K * U * (np.abs(t) @ np.abs(q)) + 64 * U * np.abs(z)
    x = np.exp(z - z.max(0))
    a = x / x.sum(0)
    ra = 2 * e_z.max(0) + 16 * U + S * U                             # relative
    o = np.einsum("sn,snd->nd", a, v)
    e_o = np.einsum("sn,snd->nd", a, np.abs(v)) * (ra + K * U)[:, None]
    out = {"rstd": (r.T, 64 * U * r.T), "logit": (z.T, e_z.T), "alpha": (a.T, a.T * ra[:, None] + 2.0 ** -126)}
    if w is None:
        out["y"] = (o, 2.0 ** -8 * np.abs(o) + e_o)
    else:
        ro = 1 / np.sqrt((o ** 2).mean(-1, keepdims=True) + eps)
        e_ro = (np.abs(o) * e_o).sum(-1, keepdims=True) / ((o ** 2).sum(-1, keepdims=True) + D * eps) + 64 * U
        y = o * ro * w
        out["y"] = (y, 2.0 ** -8 * np.abs(y) + np.abs(w) * ro * e_o + np.abs(y) * (e_ro + 4 * U))
        out["o_rstd"] = (ro[:, 0], (ro * e_ro)[:, 0])
    if dy is None:
        return out
    if w is None:
        do, e_do = dy, np.zeros_like(dy)
    else:
        h = dy * w
        c = ro ** 2 * (h * o).sum(-1, keepdims=True) / D
        e_c = ro ** 2 / D * (np.abs(h) * e_o + K * U * np.abs(h * o)).sum(-1, keepdims=True) + np.abs(c) * (2 * e_ro + 8 * U)
        do = ro * (h - o * c)
        e_do = ro * (np.abs(c) * e_o + np.abs(o) * e_c + 8 * U * (np.abs(h) + np.abs(o * c))) + np.abs(do) * e_ro
        dw = (dy * o * ro).sum(0)
        out["dw_o_f32"] = (dw, (np.abs(dy) * (ro * e_o + np.abs(o) * ro * e_ro) + np.abs(dy * o * ro) * (N + 64) * U).sum(0))
    da = np.einsum("nd,snd->sn", do, v)
    e_da = np.einsum("nd,snd->sn", e_do + K * U * np.abs(do), np.abs(v))
    m = (a * da).sum(0)
    e_m = (a * e_da + np.abs(a * da) * (ra + (S + 8) * U)).sum(0)
    dz = a * (da - m)
    e_dz = a * (e_da + e_m) + np.abs(dz) * ra + 4 * U * a * (np.abs(da) + np.abs(m))
    dv = a[..., None] * do
    e_dv = a[..., None] * (e_do + np.abs(do) * (ra[:, None] + 4 * U))
    c1, c2 = scale * dz * r, dz * z * r ** 2 / R
    dv[..., ko:ko + R] += c1[..., None] * q - c2[..., None] * t
    e_dv[..., ko:ko + R] += (abs(scale) * r * e_dz + 140 * U * np.abs(c1))[..., None] * np.abs(q)
    e_dv[..., ko:ko + R] += (np.abs(z) * r ** 2 / R * e_dz + np.abs(dz) * r ** 2 / R * e_z + 140 * U * np.abs(c2))[..., None] * np.abs(t)
    out["dvalues"] = (dv, 2.0 ** -8 * np.abs(dv) + e_dv)
    dq = np.einsum("sn,snr->r", c1, t)
    e_dq = np.einsum("sn,snr->r", abs(scale) * r * e_dz + np.abs(c1) * (N * S + 140) * U, np.abs(t))
    out["dq_f32"] = (dq, e_dq)
    return out


def check(name, got, want):
    """got: a tensor; want: (value, bound).  The worst |got - value| / bound is at most 1."""
    value, bound = want
    g = got.detach().double().cpu().numpy().reshape(value.shape)
    off = np.abs(g - value)
    bad = ~(off <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} beyond their bounds, worst "
                           f"{np.nanmax(off / np.maximum(bound, 1e-300)):.3g} times; first at {np.argwhere(bad)[0]}")
