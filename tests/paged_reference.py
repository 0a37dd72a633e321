"""Plain 64-bit forms of the paged cache's operators, on the host, over the
oracle's codec; shared by the paged tests."""
from __future__ import annotations

import numpy as np
import torch

import oracle
import workloads as W


def f64(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def rotate(x, table, positions, rotary, interleaved, inverse=False):
    """fp64 turn of x [tokens, heads, dim] (numpy), and the sums |a cos| + |b sin| of each value."""
    pos = np.clip(positions, 0, table.shape[0] - 1)
    cs, sn = table[pos, :, 0][:, None].astype(np.float64), table[pos, :, 1][:, None].astype(np.float64)
    if inverse:
        sn = -sn
    i = np.arange(rotary // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    y, size = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cs - b * sn, b * cs + a * sn
    size[..., ia], size[..., ib] = np.abs(a * cs) + np.abs(b * sn), np.abs(b * cs) + np.abs(a * sn)
    return y, size


def rotate_f32(x, table, positions, rotary, interleaved, inverse=False):
    """The turn as the kernels define it: every product and sum one fp32 rounding (numpy float32)."""
    pos = np.clip(positions, 0, table.shape[0] - 1)
    cs, sn = table[pos, :, 0][:, None], table[pos, :, 1][:, None]
    if inverse:
        sn = -sn
    i = np.arange(rotary // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    y = x.astype(np.float32)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * cs - b * sn, b * cs + a * sn
    return y


def pool_decode(blob, pages):
    """uint8 [n, H, ps, 64] -> fp64 [n, H, ps, 128]."""
    n = pages.shape[0] * pages.shape[1] * pages.shape[2]
    y = oracle.decode(blob, np.ascontiguousarray(pages).reshape(n, 64), nthreads=8)
    return f64(np.asarray(y)).reshape(*pages.shape[:3], 128)


def attend(q, kd, vd, table, kv_lens, cu_q, scale, window, max_q=None, max_kv=None):
    """(out, lse, tol_out, tol_lse) in fp64: q [T, Hq, 128] fp64, kd / vd decoded
    pools.  Tolerances, to first order: a score is a sum of 128 exact products
    in fp32, off by at most 128 2^-24 sum |q_i k_i| before the scale, and the
    scale's and the exponent's roundings add 2^-22 of its size; a weight is off
    by twice that (its own and the sum's), plus half a bf16 step (2^-8) for the
    second product and 2^-20 for exp, the sums and the division; the output's own
    rounding is half a bf16 step."""
    T, Hq, _ = q.shape
    H = kd.shape[1]
    G, ps, n_pages = Hq // H, kd.shape[2], kd.shape[0]
    out, lse = np.zeros(q.shape), np.full((T, Hq), -np.inf)
    tol, tol_lse = np.zeros(q.shape), np.zeros((T, Hq))
    written = np.zeros(T, bool)
    for b in range(len(kv_lens)):
        n, nq = int(kv_lens[b]), int(cu_q[b + 1] - cu_q[b])
        keys = max(0, min(n, table.shape[1] * ps, 1 << 30 if max_kv is None else max_kv))
        pg = table[b][np.arange(keys) // ps] if keys else np.zeros(0, int)
        bad = (pg < 0) | (pg >= n_pages)
        sl = np.arange(keys) % ps
        k = np.where(bad[:, None, None], 0.0, kd[np.where(bad, 0, pg), :, sl]) if keys else np.zeros((0, H, 128))
        v = np.where(bad[:, None, None], 0.0, vd[np.where(bad, 0, pg), :, sl]) if keys else np.zeros((0, H, 128))
        for i in range(nq if max_q is None else min(nq, max_q)):
            t, p = int(cu_q[b]) + i, n - nq + i
            written[t] = True
            lo, hi = (max(0, p - window + 1) if window else 0), min(p + 1, keys)
            if hi <= lo:
                continue
            for j in range(Hq):
                kk, vv = k[lo:hi, j // G], v[lo:hi, j // G]
                s = kk @ q[t, j] * scale
                m = s.max()
                e = np.exp(s - m)
                l = e.sum()
                w = e / l
                out[t, j] = w @ vv
                lse[t, j] = m + np.log(l)
                size = abs(scale) * (np.abs(kk) @ np.abs(q[t, j])).max()
                d = (128 * 2.0**-24 + 2.0**-22) * size
                tol[t, j] = 2.0**-8 * np.abs(out[t, j]) + (2 * d + 2.0**-8 + 2.0**-20) * (w @ np.abs(vv)) + 1e-30
                tol_lse[t, j] = d + 2.0**-20 * (1 + abs(lse[t, j]))
    return out, lse, tol * 1.01, tol_lse, written


def bits(t: torch.Tensor) -> np.ndarray:
    return W.bf16_bits(t)
