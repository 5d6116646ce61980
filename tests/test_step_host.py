"""Host-side checks (no GPU) of the bookkeeping, normed rotation and paged chunk entry points: every refusal comes back before a
CUDA call, the binding's own checks raise, and the float64 references satisfy their definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref

P, P2, P3 = 0x10000, 0x20000, 0x30000  # fake device addresses: never dereferenced
INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


def _ll(values):
    return None if values is None else (ctypes.c_longlong * len(values))(*values)


def _slots(**kw):
    a = dict(ctx=P, new=P, table=P2, stride=4, free=P3, n_free=5, count=P3, B=2, T=8, ps=16, mp=4, cu=P, pos=P, slots=P,
             lens=P, left=P)
    a.update(kw)
    return fa.lib().fa_paged_slots(a["ctx"], a["new"], a["table"], a["stride"], a["free"], a["n_free"], a["count"], a["B"],
                                   a["T"], a["ps"], a["mp"], a["cu"], a["pos"], a["slots"], a["lens"], a["left"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(count=None), INVALID), (dict(cu=None), INVALID), (dict(pos=None), INVALID), (dict(slots=None), INVALID),
    (dict(lens=None), INVALID), (dict(left=None), INVALID), (dict(ctx=P + 2), INVALID), (dict(slots=P + 4), INVALID),
    (dict(table=P2 + 1), INVALID), (dict(count=P3 + 2), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID),
    (dict(n_free=-1), INVALID), (dict(ps=0), INVALID), (dict(mp=0), INVALID), (dict(stride=3), INVALID),
    (dict(mp=1 << 20, stride=1 << 20, ps=1 << 10), INVALID), (dict(T=(1 << 30) + 1), INVALID), (dict(B=16385), UNSUPPORTED),
])
def test_slots_rejects(kw, status):
    assert _slots(**kw) == status


def _norm(backward=False, append=False, **kw):
    a = dict(q=P, k=P, qo=P2, ko=P2, dq=P, dk=P, dwq=P3, dwk=P3, strides=None, B=1, H=4, Hkv=2, N=8, d=64, dtype=fa.FA_BF16,
             wq=P3, wk=P3, wt=fa.FA_FP32, eps=1e-6, pos=P3, shared=0, freqs=P3, axes=None, n_axes=1, rot=64, inter=0, ws=None,
             wsb=0, v=P, kc=P2, vc=P2, slots=P3, T=4, pages=8, ps=16)
    a.update(kw)
    L = fa.lib()
    tail = (a["wq"], a["wk"], a["wt"], a["eps"], a["pos"])
    if append:
        return L.fa_paged_append_norm(a["k"], a["v"], a["q"], a["qo"], a["kc"], a["vc"], None, None, a["slots"], a["T"], a["H"],
                                      a["Hkv"], a["d"], a["pages"], a["ps"], *tail, a["freqs"], a["axes"], a["n_axes"],
                                      a["rot"], a["inter"], None)
    rest = (a["shared"], a["freqs"], a["axes"], a["n_axes"], a["rot"], a["inter"])
    sizes = (a["B"], a["H"], a["Hkv"], a["N"], a["d"], a["dtype"])
    if backward:
        return L.fa_norm_rope_bwd(a["dq"], a["dk"], a["q"], a["k"], a["qo"], a["ko"], a["dwq"], a["dwk"], _ll(a["strides"]),
                                  *sizes, *tail, *rest, a["ws"], a["wsb"], None)
    return L.fa_norm_rope(a["q"], a["k"], a["qo"], a["ko"], _ll(a["strides"]), *sizes, *tail, *rest, None)


COMMON = [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(q=P + 8), INVALID), (dict(wq=None), INVALID), (dict(wk=None), INVALID),
    (dict(wq=P3 + 2), INVALID), (dict(wk=P3 + 1, wt=fa.FA_BF16), INVALID), (dict(wt=7), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(pos=None), INVALID), (dict(freqs=None), INVALID),
    (dict(rot=0), INVALID), (dict(rot=72), INVALID), (dict(rot=24), UNSUPPORTED), (dict(n_axes=0), INVALID),
    (dict(n_axes=9), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(H=0), INVALID), (dict(inter=2), INVALID),
]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(k=None), INVALID), (dict(ko=None), INVALID), (dict(Hkv=0), INVALID),
                                                (dict(dtype=5), UNSUPPORTED), (dict(N=0), INVALID), (dict(shared=2), INVALID)])
def test_norm_rope_rejects(kw, status):
    assert _norm(**kw) == status
    assert _norm(backward=True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dwq=None), INVALID), (dict(dwk=None), INVALID),
    (dict(dwq=P3 + 2), INVALID), (dict(ws=P + 4), INVALID), (dict(strides=[512, 64, 64] * 5 + [512, 64, 60]), INVALID),
    (dict(strides=[512, 64, 64] * 4 + [512, -64, 64] * 2), INVALID), (dict(strides=[512, 64, 64] * 2 + [512, 64, 0] + [512, 64, 64] * 3), INVALID),
])
def test_norm_rope_bwd_rejects(kw, status):
    assert _norm(backward=True, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
                                                (dict(T=-1), INVALID), (dict(pages=0), INVALID)])
def test_append_norm_rejects(kw, status):
    assert _norm(append=True, **kw) == status


def _fwd(**kw):
    a = dict(q=P, kc=P, vc=P, o=P2, pt=P3, stride=None, cu=P3, lens=P3, T=9, B=2, H=8, Hkv=2, d=64, pages=8, ps=16, mp=4,
             qs=None, cs=None, scale=0.125, window=0, sinks=0, ws=None, wsb=0, lse=None)
    a.update(kw)
    if a["stride"] is None:
        a["stride"] = a["mp"]
    return fa.lib().fa_fwd_paged(a["q"], a["kc"], a["vc"], a["o"], a["pt"], a["stride"], a["cu"], a["lens"], a["T"], a["B"],
                                 a["H"], a["Hkv"], a["d"], a["pages"], a["ps"], a["mp"], _ll(a["qs"]), _ll(a["cs"]), a["scale"],
                                 a["window"], a["sinks"], a["ws"], a["wsb"], a["lse"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(o=None), INVALID), (dict(pt=None), INVALID),
    (dict(cu=None), INVALID), (dict(lens=None), INVALID), (dict(q=P + 8), INVALID), (dict(vc=P + 2), INVALID), (dict(pt=P3 + 2), INVALID),
    (dict(cu=P3 + 1), INVALID), (dict(lse=P3 + 2), INVALID), (dict(ws=P + 8), INVALID), (dict(T=-1), INVALID), (dict(B=-1), INVALID),
    (dict(H=0), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(ps=0), INVALID),
    (dict(mp=0), INVALID), (dict(stride=3), INVALID), (dict(mp=1 << 20, ps=1 << 10), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=3e38), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(H=129, Hkv=1), UNSUPPORTED), (dict(B=16385), UNSUPPORTED), (dict(T=1 << 29, H=64), INVALID),
    (dict(T=1 << 16, H=8, Hkv=1, B=200, mp=1 << 16, ps=1 << 13), INVALID),
    (dict(qs=[512, 60]), INVALID), (dict(qs=[512, 0]), INVALID), (dict(qs=[0, 64]), INVALID), (dict(qs=[-512, 64]), INVALID),
    (dict(qs=[64, 1024]), INVALID), (dict(cs=[2048, 1024, 60]), INVALID), (dict(cs=[0, 1024, 64]), INVALID),
])
def test_fwd_paged_rejects(kw, status):
    assert _fwd(**kw) == status


def test_workspace_bytes_of_bad_arguments():
    for bad in ((0, 2, 8, 2, 64), (9, 0, 8, 2, 64), (9, 2, 8, 3, 64), (9, 2, 8, 2, 96), (9, 2, 129, 1, 64), (9, 16385, 8, 2, 64)):
        assert fa.fa_fwd_paged_workspace_bytes(*bad) == 0
    assert fa.fa_norm_rope_bwd_workspace_bytes(96) == 0


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16), torch.ones(64)
    pos, freqs = torch.zeros(8, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    i = torch.zeros(1, dtype=torch.int32)
    c, t = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.fa_norm_rope(x, x, w, w, pos, freqs), lambda: fa.fa_norm_rope_bwd(x, x, x, x, w, w, pos, freqs),
                 lambda: fa.fa_paged_slots(i, i, i.view(1, 1), i, i, 16, 4),
                 lambda: fa.fa_fwd_paged(t, c, c, i.view(1, 1), i, i),
                 lambda: fa.fa_paged_append(t, t, c, c, torch.zeros(3, dtype=torch.int64), k_weight=w)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        fa.fa_fwd_paged(None, c, c, i, i, i)
    with pytest.raises(TypeError):
        fa.fa_norm_rope(x, x, None, w, pos, freqs)


# ------------------------------------------------------------------------------------------ the references

def test_norm_reference_gradient_is_the_difference():
    rng = np.random.default_rng(1)
    x, w, dy = rng.normal(size=(5, 3, 64)), rng.normal(size=64), rng.normal(size=(5, 3, 64))
    freqs, axes, pos = 10000.0 ** (-np.arange(16) / 16), np.arange(16) % 2, rng.integers(0, 1000, (2, 5))
    for inter in (False, True):
        args = (1e-5, pos, freqs, axes, inter)
        dx, dw, tol, tol_w = ref.norm_rope_bwd(dy, x, w, *args)
        h, ex, ew = 1e-5, rng.normal(size=x.shape), rng.normal(size=64)
        up, down = (ref.norm_rope(x + s * h * ex, w + s * h * ew, *args)[0] for s in (1, -1))
        assert abs(((up - down) * dy).sum() / (2 * h) - (dx * ex).sum() - (dw * ew).sum()) < 1e-7
        assert (tol < 1e-4).all() and (tol_w < 1e-3).all()


def test_attention_reference_is_the_decodes_definition():
    """A chunk's row equals one query over the keys it sees."""
    import paged_ref

    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(6, 64)), rng.normal(size=(30, 64)), rng.normal(size=(30, 64))
    for window, sinks in ((0, 0), (4, 0), (5, 3), (1, 0)):
        seen = ref.visible(24, 6, window, sinks)
        o, lse, _, _ = ref.attend(q, k, v, seen, 0.125)
        for i in range(6):
            at = [j for j in range(30) if j <= 24 + i and (not window or j > 24 + i - window or j < sinks)]
            ro, rl, _, _ = paged_ref.attend(q[i], k[at], v[at], 0.125)
            assert np.allclose(o[i], ro, atol=1e-13) and abs(lse[i] - rl) < 1e-13


def test_slots_reference_by_hand():
    cu, pos, slots, lens, left, table, failed = ref.slots([3, 0, 8], [2, 0, 1], [[9, 0], [0, 0], [5, 6]], [1, 2, 7], 3, 4, 4)
    assert (cu, pos, slots, lens, left, failed) == ([0, 2, 2, 3], [3, 4, 0, 0], [39, 28, -1, -1], [5, 0, -1], 2, True)
    assert table == [[9, 7], [0, 0], [5, 6]]
