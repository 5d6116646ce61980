"""Float64 references of the position and paged-cache operators, and the bounds their GPU results are held to.

The references are the definitions, in numpy, one token or sequence at a time; they share no code with the library.

Bounds (each counts the roundings of the computation; half steps u: bf16 2^-8, fp32 2^-24, relative):
  rotation   cos and sin: the phase's upper 32 bits become an fp32 number of half turns (at most pi 2^-25 rad off) and
             sincospif adds at most 2 ulp: together below 2.2e-7.  Two products and a sum in fp32 add 3 u_fp32.  So
             |dy| <= 4.5e-7 (|x1| + |x2|), plus |x1| + |x2| times |pos| f 2^-51 for the frequency's double rounding (in
             the kernel and here), plus u |y| for the output's rounding.
  decode     a score is a sum of d exact bf16 products in fp32, then scaled: off by at most
             ds = (d + 4) u_fp32 |scale| sum |q_i k_i|.  P is off by ds + 2^-20 relative (ex2.approx and its argument's
             rounding) and rounded to bf16, u_bf16, before P V: |dO| <= (u_bf16 + 2 ds + 2^-19 + n u_fp32) sum p |v|
             + u_bf16 |O|.  LSE: a thread adds at most n/16 + 64 terms in turn: |dLSE| <= ds + (n/16 + 64) u_fp32 +
             2^-20 + 4 u_fp32 |LSE|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def pairs(rot: int, interleaved: bool):
    n = rot // 2
    if interleaved:
        return np.arange(0, rot, 2), np.arange(1, rot, 2)
    return np.arange(n), np.arange(n, rot)


def rotate(x: np.ndarray, pos: np.ndarray, freqs: np.ndarray, axes: np.ndarray, interleaved: bool, inverse=False):
    """x [..., heads, d] with pos [A, ...] (one position per axis for a row of heads); returns (y, bound without the
    output's rounding)."""
    rot = 2 * len(freqs)
    i1, i2 = pairs(rot, interleaved)
    y, tol = x.copy(), np.zeros_like(x)
    for i in range(len(freqs)):
        p = pos[axes[i]].astype(np.float64)[..., None]
        phi = p * freqs[i] * (-1.0 if inverse else 1.0)
        x1, x2 = x[..., i1[i]], x[..., i2[i]]
        y[..., i1[i]] = x1 * np.cos(phi) - x2 * np.sin(phi)
        y[..., i2[i]] = x1 * np.sin(phi) + x2 * np.cos(phi)
        t = (np.abs(x1) + np.abs(x2)) * (4.5e-7 + np.abs(p) * abs(freqs[i]) * 2.0 ** -51)
        tol[..., i1[i]] = tol[..., i2[i]] = t
    return y, tol


def check_rotated(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray, name: str):
    g = f64(got)
    bad = np.abs(g - ref) > U[got.dtype] * np.abs(ref) + tol
    assert np.isfinite(g).all(), f"{name}: not finite"
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside the bound, worst {np.abs(g - ref).max():.3e}"
    same = tol == 0.0  # elements that are copied
    assert np.array_equal(g[same], ref[same]), f"{name}: a copied element changed"


def sequence_rows(cache: torch.Tensor, pages, n: int, h: int) -> np.ndarray:
    """Rows 0 .. n-1 of a sequence whose pages are listed, of key/value head h: [n, d]."""
    ps = cache.shape[2]
    at = torch.arange(n)
    pg = torch.as_tensor(np.asarray(pages, dtype=np.int64))[at // ps]
    return f64(cache[pg.to(cache.device), h, (at % ps).to(cache.device)])


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """One query [d] over k, v [n, d]: (o, lse, bound of o without the output's rounding, bound of lse)."""
    n, d = k.shape
    if n == 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    s = (k @ q) * scale
    m = s.max()
    e = np.exp(s - m)
    total = e.sum()
    p = e / total
    lse = m + math.log(total)
    u, ub = 2.0 ** -24, 2.0 ** -8
    ds = (d + 4) * u * abs(scale) * (np.abs(k) @ np.abs(q)).max()
    tol_o = (ub + 2 * ds + 2.0 ** -19 + n * u) * (p @ np.abs(v))
    return p @ v, lse, tol_o, ds + (n / 16 + 64) * u + 2.0 ** -20 + 4 * u * abs(lse)


def check_decode(q, kc, vc, o, lse, tables, lens, scale, name, prefix=(), prefix_len=0, heads=None, seqs=None):
    """Checks o [B,H,d] (and lse [B,H]) against the definition.  tables[b]: page ids of sequence b; a negative length
    sees nothing."""
    B, H, d = o.shape
    G = H // kc.shape[1]
    og, lg = f64(o), None if lse is None else f64(lse)
    worst = 0.0
    for hk in sorted({h // G for h in (heads if heads is not None else range(H))}):
        pk = sequence_rows(kc, prefix, prefix_len, hk) if prefix_len else np.zeros((0, d))
        pv = sequence_rows(vc, prefix, prefix_len, hk) if prefix_len else np.zeros((0, d))
        for b in (seqs if seqs is not None else range(B)):
            n = int(lens[b])
            if n < 0:
                k, v = np.zeros((0, d)), np.zeros((0, d))
            else:
                k = np.concatenate([pk, sequence_rows(kc, tables[b], n, hk)]) if n else pk
                v = np.concatenate([pv, sequence_rows(vc, tables[b], n, hk)]) if n else pv
            for h in range(hk * G, (hk + 1) * G):
                if heads is not None and h not in heads:
                    continue
                ro, rl, to, tl = attend(f64(q.reshape(B, H, d)[b, h]), k, v, scale)
                err, lim = np.abs(og[b, h] - ro), to + 2.0 ** -8 * np.abs(ro)
                assert (err <= lim).all(), (f"{name}: o of sequence {b} head {h} (length {n}) off by {err.max():.3e}, "
                                            f"bound {lim[err.argmax()]:.3e}")
                if k.shape[0]:
                    worst = max(worst, (err / np.maximum(lim, 1e-30)).max())
                if lg is not None:
                    if k.shape[0] == 0:
                        assert lg[b, h] == -np.inf, f"{name}: lse of an empty sequence"
                    else:
                        assert abs(lg[b, h] - rl) <= tl, f"{name}: lse of sequence {b} head {h}: {lg[b, h]} not {rl}"
    print(f"[parity] {name}: worst error/bound {worst:.2f}")


def paged_cache(pages: int, Hkv: int, ps: int, d: int, device, seed: int, layout: str = "head"):
    """(k_cache, v_cache) of shape [pages, Hkv, ps, d], N(0,1).  layout: "head" contiguous; "row" [pages, ps, Hkv, d];
    "one" both interleaved in one buffer [pages, 2, ps, Hkv, d]; "odd" padded rows, heads and pages
    (strides that are not multiples of one another)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g, device=device).to(torch.bfloat16)

    if layout == "head":
        return draw(pages, Hkv, ps, d), draw(pages, Hkv, ps, d)
    if layout == "row":
        return draw(pages, ps, Hkv, d).transpose(1, 2), draw(pages, ps, Hkv, d).transpose(1, 2)
    if layout == "odd":
        row, head = d + 8, ps * (d + 8) + 24
        page = Hkv * head + 40
        return tuple(draw(pages * page + 64)[16:].as_strided((pages, Hkv, ps, d), (page, head, row, 1)) for _ in range(2))
    both = draw(pages, 2, ps, Hkv, d)
    return both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)


def deal_pages(lens, ps: int, seed: int, extra: int = 0, spare: int = 2):
    """Shuffled page ids: (list of each sequence's pages, `extra` further pages, number of pages)."""
    need = [max(0, -(-int(n) // ps)) for n in lens]
    total = sum(need) + extra + spare
    order = np.random.default_rng(seed).permutation(total)
    out, at = [], 0
    for n in need:
        out.append(order[at:at + n])
        at += n
    return out, order[at:at + extra], total


def page_table(tables, device, width=None, junk=-7):
    """The tables as an int32 tensor [B, width]; entries past a sequence's pages are junk."""
    width = width or max(1, max((len(t) for t in tables), default=1))
    out = np.full((len(tables), width), junk, dtype=np.int32)
    for b, t in enumerate(tables):
        out[b, :len(t)] = t
    return torch.as_tensor(out, device=device)


def spoil_unused(kc, vc, tables, lens, prefix=(), prefix_len=0):
    """NaN and infinities into every cache row that no sequence sees."""
    pages, _, ps, _ = kc.shape
    seen = torch.zeros(pages, ps, dtype=torch.bool)
    for t, n in [*zip(tables, lens), (prefix, prefix_len)]:
        for i in range(max(0, int(n))):
            seen[int(t[i // ps]), i % ps] = True
    free = (~seen).to(kc.device)[:, None, :, None]
    kc.copy_(torch.where(free, torch.tensor(float("nan"), dtype=kc.dtype, device=kc.device), kc))
    vc.copy_(torch.where(free, torch.tensor(float("inf"), dtype=vc.dtype, device=vc.device), vc))
