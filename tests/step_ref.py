"""Float64 references of the step operators (bookkeeping, head norms with rotation, paged chunk attention), and the bounds
their GPU results are held to.  Definitions in numpy; they share no code with the library.

Bounds (half steps u: bf16 2^-8, fp32 2^-24, relative):
  norm       mean(x^2) is a sum of d squares in fp32 in some order: off by at most d u relative; the root and its
             reciprocal halve that and add 2^-22 (rsqrtf); three products follow: e = (d/2 + 4) u + 2^-22 for w r x.  The
             rotation adds what paged_ref.rotate says, on values that are off by e: (|z1| + |z2|) (e + 4.5e-7 + pos f 2^-51).
  its bwd    g = R^-1 dy is off by tg = (|dy1| + |dy2|) (4.5e-7 + pos f 2^-51).  m = mean(w g u) is off by mean(|w| tg |u|) +
             (2 d u + 2 e) mean(|w g u|).  dx = r (w g - u m): r (|w| tg + |u| dm + (e + 4 u) (|w g| + |u m|)) with the r in
             front off by e too.  dw: n terms g u, each off by tg |u| + (e + 2 u) |g u|, added in fp32: n u sum |g u| more.
             All plus the output's rounding.
  attention  paged_ref's for the decode (P may be rounded to bf16 before P V): |dO| <= (u_bf16 + 2 ds + 2^-19 + n u) sum p |v|
             + u_bf16 |O| with ds = (d + 4) u |scale| max sum |q k|; |dLSE| <= ds + (n/16 + 64) u + 2^-20 + 4 u |LSE|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from paged_ref import U, f64, pairs, rotate

U32 = 2.0 ** -24


# ------------------------------------------------------------------------------------------ bookkeeping

def slots(ctx, new, table, free, count, ps, T):
    """One sequence at a time, by the rules of the entry point: (cu, positions, slots, lens, left, table, any failed)."""
    B, width = len(ctx), len(table[0]) if len(table) else 1
    table = [list(r) for r in table]
    cu, pos, out, lens = [0], [0] * T, [-1] * T, []
    top = count if 0 <= count <= len(free) else 0
    dealt, at, failed, left = 0, 0, not 0 <= count <= len(free), top
    for b in range(B):
        n, c = max(0, int(new[b])), int(ctx[b])
        first, at = at, at + n
        cu.append(min(at, T))
        if n == 0:
            lens.append(c)
            continue
        ok = c >= 0 and at <= T and c + n <= width * ps
        if ok:
            held, need = -(-c // ps), -(-(c + n) // ps) - -(-c // ps)
            base, dealt = dealt, dealt + need
            ok = need == 0 or dealt <= top
        if not ok:
            failed = True
            lens.append(-1)
            continue
        for i in range(need):
            table[b][held + i] = free[top - 1 - base - i]
        if need:
            left = top - dealt
        for i in range(n):
            p = c + i
            pos[first + i] = p
            page = table[b][p // ps]
            out[first + i] = page * ps + p % ps if page >= 0 else -1
        lens.append(c + n)
    return cu, pos, out, lens, left, table, failed


# ------------------------------------------------------------------------------------------ norms

def norm_rope(x, w, eps, pos=None, freqs=None, axes=None, interleaved=False):
    """x [..., heads, d], pos [A, ...]; returns (y, bound without the output's rounding)."""
    d = x.shape[-1]
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    e = (d / 2 + 4) * U32 + 2.0 ** -22
    if freqs is None or len(freqs) == 0:
        return z, e * np.abs(z)
    y, tol = rotate(z, pos, freqs, axes, interleaved)
    i1, i2 = pairs(2 * len(freqs), interleaved)
    extra = e * np.abs(z)
    both = e * (np.abs(z[..., i1]) + np.abs(z[..., i2]))
    extra[..., i1] = extra[..., i2] = both
    return y, tol + extra


def norm_rope_bwd(dy, x, w, eps, pos=None, freqs=None, axes=None, interleaved=False):
    """(dx, dw, bound of dx without the output's rounding, bound of dw); heads and d are the last axes."""
    d = x.shape[-1]
    if freqs is None or len(freqs) == 0:
        g, tg = dy, np.zeros_like(dy)
    else:
        g, tg = rotate(dy, pos, freqs, axes, interleaved, inverse=True)
    e = (d / 2 + 4) * U32 + 2.0 ** -22
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u, wg = x * r, w * g
    m = (wg * u).mean(-1, keepdims=True)
    dx = r * (wg - u * m)
    dm = (np.abs(w) * tg * np.abs(u)).mean(-1, keepdims=True) + (2 * d * U32 + 2 * e) * np.abs(wg * u).mean(-1, keepdims=True)
    tol = r * (np.abs(w) * tg + np.abs(u) * dm + (2 * e + 4 * U32) * (np.abs(wg) + np.abs(u * m)))
    rest = tuple(range(x.ndim - 1))
    n = x.size // d
    terms = np.abs(g * u)
    tol_w = (tg * np.abs(u) + (e + 2 * U32) * terms).sum(rest) + n * U32 * terms.sum(rest)
    return dx, (g * u).sum(rest), tol, tol_w


def check(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray, name: str):
    g = f64(got)
    assert g.shape == ref.shape, f"{name}: shape {g.shape} not {ref.shape}"
    bad = ~(np.abs(g - ref) <= U[got.dtype] * np.abs(ref) + tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside the bound, worst {np.nanmax(np.abs(g - ref)):.3e}"


# ------------------------------------------------------------------------------------------ attention

def visible(ctx, n, window, sinks):
    """[n, ctx + n] truth values: which keys each new token sees."""
    p = np.arange(ctx, ctx + n)[:, None]
    j = np.arange(ctx + n)[None, :]
    seen = j <= p
    return seen & ((j > p - window) | (j < sinks)) if window else seen


def attend(q, k, v, seen, scale):
    """q [n, d] over k, v [N, d] where seen [n, N]: (o, lse, their bounds)."""
    n, d = q.shape
    with np.errstate(invalid="ignore"):
        s = np.where(seen, (q @ k.T) * scale, -np.inf)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    total = e.sum(-1, keepdims=True)
    p = e / total
    N = seen.sum(-1, keepdims=True)
    ds = (d + 4) * U32 * abs(scale) * np.where(seen, np.abs(q) @ np.abs(k).T, 0).max(-1, keepdims=True)
    o = p @ v
    tol = (2.0 ** -8 + 2 * ds + 2.0 ** -19 + N * U32) * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(o)
    lse = (m + np.log(total))[:, 0]
    return o, lse, tol, ds[:, 0] + (N[:, 0] / 16 + 64) * U32 + 2.0 ** -20 + 4 * U32 * np.abs(lse)


def check_fwd_paged(q, kc, vc, tables, lens, news, o, lse, name, scale=None, window=0, sinks=0, seqs=None, heads=None):
    """Checks o [T,H,d] and lse [T,H] of the sequences against the definition; tables[b]: its page ids."""
    T, H, d = o.shape
    Hkv, ps = kc.shape[1], kc.shape[2]
    G = H // Hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    og, qg, lg = f64(o), f64(q), None if lse is None else f64(lse)
    first, worst = 0, 0.0
    for b, n in enumerate(news):
        if n and (seqs is None or b in seqs):
            ctx = lens[b] - n
            seen = visible(ctx, n, window, sinks)
            at = np.flatnonzero(seen.any(0))  # keys that no token sees may lie in pages that are gone
            pg = torch.as_tensor(np.asarray(tables[b], dtype=np.int64)[at // ps]).to(kc.device)
            row = torch.as_tensor(at % ps).to(kc.device)
            for hk in range(Hkv):
                k, v = f64(kc[pg, hk, row]), f64(vc[pg, hk, row])
                for h in range(hk * G, (hk + 1) * G):
                    if heads is not None and h not in heads:
                        continue
                    ro, rl, to, tl = attend(qg[first:first + n, h], k, v, seen[:, at], scale)
                    err = np.abs(og[first:first + n, h] - ro)
                    assert (err <= to).all(), (f"{name}: o of sequence {b} head {h} off by {np.nanmax(err):.3e} "
                                               f"({(~(err <= to)).sum()} of {err.size} outside)")
                    worst = max(worst, (err / to).max())
                    if lg is not None:
                        le = np.abs(lg[first:first + n, h] - rl)
                        assert (le <= tl).all(), f"{name}: lse of sequence {b} head {h} off by {np.nanmax(le):.3e}"
        first += n
    print(f"[parity] {name}: worst error/bound {worst:.2f}")
