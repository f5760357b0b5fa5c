"""Float64 definitions of the score-modified attention, the rotary positions
and the 8-bit cache operators.

  x_ij = scale q_i.k_j;  cap > 0: x <- cap tanh(x / cap);  x <- x - slope_h |i - j|
  row i sees keys lo_i <= j < hi_i (and those inside the window);
  O_i = sum_j softmax(x_i)_j v_j, LSE_i = log sum_j exp(x_ij); a row that sees
  nothing has O = 0 and LSE = -inf, and no gradient.

Plain loops over batch and heads; nothing is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64, _group
from .fp8 import BLOCK, e4m3_decode, e4m3_encode, pow2_exponent


def mask_rows(b_, n, doc_ids=None, prefix_lens=None, causal=True):
    """[B, N, 2] int64: the keys [lo, hi) that each row sees, by walking the rows."""
    out = np.zeros((b_, n, 2), dtype=np.int64)
    for b in range(b_):
        i = 0
        while i < n:
            j = i + 1
            while j < n and (doc_ids is None or doc_ids[b][j] == doc_ids[b][i]):
                j += 1
            if doc_ids is None or doc_ids[b][i] >= 0:
                for r in range(i, j):
                    hi = j
                    if causal:
                        hi = r + 1
                        if prefix_lens is not None:
                            hi = max(hi, min(j, int(prefix_lens[b])))
                    out[b, r] = (i, hi)
            i = j
    return out


def _visible(n, ranges, window):
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    vis = np.ones((n, n), dtype=bool) if ranges is None else (j >= ranges[:, :1]) & (j < ranges[:, 1:])
    if window[0] >= 0:
        vis &= j >= i - window[0]
    if window[1] >= 0:
        vis &= j <= i + window[1]
    return vis


def _head(q, k, v, scale, cap, slope, vis):
    """One head: O, LSE, P and the derivative of the score by scale q.k."""
    x = scale * (q @ k.T)
    dx = np.ones_like(x)
    if cap > 0:
        t = np.tanh(x / cap)
        x, dx = cap * t, 1.0 - t * t
    n, m = x.shape
    x = x - slope * np.abs(np.arange(n)[:, None] - np.arange(m)[None, :])
    x = np.where(vis, x, -np.inf)
    mx = np.where(vis.any(1), x.max(1), 0.0)[:, None]
    e = np.exp(x - mx)
    l = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (mx + np.log(l))[:, 0]
    p = e / np.where(l > 0, l, 1.0)
    return p @ v, lse, p, dx


def forward(q, k, v, scale, ranges=None, window=(-1, -1), cap=0.0, slopes=None):
    """Dense [B, Hq, N, d], [B, Hkv, N, d] -> O, LSE."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    b_, hq, n, _ = q.shape
    g = _group(hq, k.shape[1])
    o, lse = np.empty_like(q), np.empty((b_, hq, n))
    for b in range(b_):
        vis = _visible(n, None if ranges is None else ranges[b], window)
        for h in range(hq):
            s = 0.0 if slopes is None else float(slopes[h])
            o[b, h], lse[b, h], _, _ = _head(q[b, h], k[b, h // g], v[b, h // g], scale, cap, s, vis)
    return o, lse


def backward(q, k, v, do, scale, ranges=None, window=(-1, -1), cap=0.0, slopes=None):
    """Gradients of sum(dO o O): dQ, and dK, dV summed over the query heads of a group."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    b_, hq, n, _ = q.shape
    g = _group(hq, k.shape[1])
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(b_):
        vis = _visible(n, None if ranges is None else ranges[b], window)
        for h in range(hq):
            s = 0.0 if slopes is None else float(slopes[h])
            o, _, p, dx = _head(q[b, h], k[b, h // g], v[b, h // g], scale, cap, s, vis)
            dp = do[b, h] @ v[b, h // g].T
            ds = p * (dp - (do[b, h] * o).sum(1, keepdims=True)) * dx * scale
            dq[b, h] = ds @ k[b, h // g]
            dk[b, h // g] += ds.T @ q[b, h]
            dv[b, h // g] += p.T @ do[b, h]
    return dq, dk, dv


def rotate(x, cos, sin, interleaved=False, inverse=False):
    """x [..., N, d] turned by cos, sin [..., N, rot/2] (broadcast over the leading axes)."""
    x = _f64(x).copy()
    c, s = _f64(cos), _f64(sin)
    half = c.shape[-1]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., first].copy(), x[..., second].copy()
    s = -s if inverse else s
    x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x


def rotate_fp32(x, cos, sin, interleaved=False):
    """The same in float32, every product and sum rounded on its own."""
    x = np.asarray(x, dtype=np.float32).copy()
    c, s = np.asarray(cos, dtype=np.float32), np.asarray(sin, dtype=np.float32)
    half = c.shape[-1]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x


def append_block(codes, factor, held, rows):
    """One block of one head: its first ``held`` rows of E4M3 codes with ``factor``, and new float rows behind
    them -> (codes of held + len(rows) rows, factor)."""
    old = e4m3_decode(codes[:held]) * float(factor) if held else np.zeros((0, rows.shape[-1]))
    both = np.concatenate([old, _f64(rows)])
    e = int(pow2_exponent(np.abs(both).max()))
    return e4m3_encode(both * 2.0 ** e), np.float32(2.0 ** -e)


def append_sequence(codes, factors, held, rows):
    """A sequence's [H, Nmax, d] codes and [H, blocks] factors after appending rows [H, n, d] behind ``held``."""
    codes, factors = codes.copy(), factors.copy()
    n = rows.shape[1]
    for h in range(codes.shape[0]):
        for t in range(held // BLOCK, -(-(held + n) // BLOCK) if n else 0):
            lo, hi = max(held, t * BLOCK), min(held + n, (t + 1) * BLOCK)
            c, f = append_block(codes[h, t * BLOCK:(t + 1) * BLOCK], factors[h, t], lo - t * BLOCK,
                                rows[h, lo - held:hi - held])
            codes[h, t * BLOCK:hi] = c
            factors[h, t] = f
    return codes, factors


def decode(q, k, v, lens, scale, cap=0.0, slopes=None, window_left=-1):
    """q [B, Hq, d], float k, v [B, Hkv, Nmax, d]: token L - 1 of each sequence -> O, LSE, and sum_j p_j |v_j|."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    b_, hq, d = q.shape
    g = _group(hq, k.shape[1])
    o, lse, mag = np.zeros((b_, hq, d)), np.full((b_, hq), -np.inf), np.zeros((b_, hq, d))
    for b in range(b_):
        n = int(lens[b])
        if n == 0:
            continue
        lo = max(0, n - 1 - window_left) if window_left >= 0 else 0
        for h in range(hq):
            x = scale * (k[b, h // g, lo:n] @ q[b, h])
            if cap > 0:
                x = cap * np.tanh(x / cap)
            if slopes is not None:
                x = x - float(slopes[h]) * np.arange(n - 1 - lo, -1, -1)
            e = np.exp(x - x.max())
            lse[b, h] = x.max() + np.log(e.sum())
            o[b, h] = e @ v[b, h // g, lo:n] / e.sum()
            mag[b, h] = e @ np.abs(v[b, h // g, lo:n]) / e.sum()
    return o, lse, mag
