"""Host-side checks (no GPU) of the position and paged-cache entry points: every refusal comes back before a CUDA
call, the Python binding's own checks raise, and the float64 references of the GPU tests satisfy their definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import paged_ref as ref

# Fake device addresses: never dereferenced, every call below is refused before anything is launched.
P, P2, P3 = 0x10000, 0x20000, 0x30000
BIG = 1 << 30


def _ll(values):
    return None if values is None else (ctypes.c_longlong * len(values))(*values)


def _rope(**kw):
    a = dict(q=P, k=P, qo=P2, ko=P2, strides=None, B=1, H=4, Hkv=2, N=8, d=64, dtype=fa.FA_BF16, pos=P3, shared=0,
             freqs=P3, axes=None, n_axes=1, rot=64, inter=0, inverse=0)
    a.update(kw)
    return fa.lib().fa_rope(a["q"], a["k"], a["qo"], a["ko"], _ll(a["strides"]), a["B"], a["H"], a["Hkv"], a["N"],
                            a["d"], a["dtype"], a["pos"], a["shared"], a["freqs"], a["axes"], a["n_axes"], a["rot"],
                            a["inter"], a["inverse"], None)


INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID),
    (dict(Hkv=0), INVALID), (dict(k=None, ko=None), INVALID), (dict(q=P + 8), INVALID), (dict(ko=P2 + 2), INVALID),
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(N=0), INVALID), (dict(Hkv=-1), INVALID),
    (dict(pos=None), INVALID), (dict(freqs=None), INVALID), (dict(freqs=P3 + 4), INVALID), (dict(pos=P3 + 2), INVALID),
    (dict(axes=P3 + 2), INVALID), (dict(n_axes=0), INVALID), (dict(n_axes=9), UNSUPPORTED), (dict(rot=0), INVALID),
    (dict(rot=72), INVALID), (dict(rot=24), UNSUPPORTED), (dict(inter=2), INVALID), (dict(inverse=-1), INVALID),
    (dict(shared=3), INVALID), (dict(d=96), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED),
    (dict(B=1 << 20, N=1 << 20), INVALID),
    (dict(strides=[512, 64, 64] * 3 + [512, 64, 60]), INVALID), (dict(strides=[512, 64, -64] * 4), INVALID),
    (dict(strides=[512, 64, 64] * 2 + [0, 64, 64] + [512, 64, 64], B=2), INVALID),
    (dict(strides=[512, 64, 64] * 3 + [512, 64, 0], N=2), INVALID), (dict(H=1 << 25), INVALID),
])
def test_rope_rejects(kw, status):
    assert _rope(**kw) == status


def _append(**kw):
    a = dict(k=P, v=P, q=P, qo=P2, kc=P2, vc=P2, ins=None, cs=None, slots=P3, T=4, H=4, Hkv=2, d=64, pages=8, ps=16,
             pos=P3, freqs=P3, axes=None, n_axes=1, rot=64, inter=0)
    a.update(kw)
    return fa.lib().fa_paged_append(a["k"], a["v"], a["q"], a["qo"], a["kc"], a["vc"], _ll(a["ins"]), _ll(a["cs"]),
                                    a["slots"], a["T"], a["H"], a["Hkv"], a["d"], a["pages"], a["ps"], a["pos"],
                                    a["freqs"], a["axes"], a["n_axes"], a["rot"], a["inter"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(slots=None), INVALID), (dict(slots=P3 + 4), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(H=0), INVALID), (dict(q=None, qo=None), INVALID), (dict(T=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(pages=0), INVALID), (dict(ps=0), INVALID), (dict(kc=P2 + 8), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(rot=0), INVALID), (dict(pos=None), INVALID), (dict(freqs=None), INVALID), (dict(rot=80), INVALID),
    (dict(rot=40), UNSUPPORTED), (dict(ins=[128, 60, 128, 64, 256, 64]), INVALID), (dict(cs=[2048, 1024, 4]), INVALID),
    (dict(cs=[2048, -1024, 64]), INVALID), (dict(Hkv=1 << 24), INVALID),
])
def test_append_rejects(kw, status):
    assert _append(**kw) == status


def _decode(**kw):
    a = dict(q=P, kc=P, vc=P, o=P2, pp=None, plen=0, pt=P3, stride=None, lens=P3, B=2, H=8, Hkv=2, d=64, pages=8, ps=16,
             mp=4, cs=None, scale=0.125, ws=None, wsb=0, lse=None)
    a.update(kw)
    if a["stride"] is None:
        a["stride"] = a["mp"]
    return fa.lib().fa_decode_paged_prefix(a["q"], a["kc"], a["vc"], a["o"], a["pp"], a["plen"], a["pt"], a["stride"],
                                           a["lens"], a["B"], a["H"], a["Hkv"], a["d"], a["pages"], a["ps"], a["mp"],
                                           _ll(a["cs"]), a["scale"], a["ws"], a["wsb"], a["lse"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(o=None), INVALID),
    (dict(pt=None), INVALID), (dict(lens=None), INVALID), (dict(q=P + 8), INVALID), (dict(vc=P + 2), INVALID),
    (dict(pt=P3 + 2), INVALID), (dict(lens=P3 + 1), INVALID), (dict(lse=P3 + 2), INVALID), (dict(ws=P + 8), INVALID),
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=3), INVALID), (dict(pages=0), INVALID),
    (dict(ps=0), INVALID), (dict(mp=0), INVALID), (dict(stride=3), INVALID), (dict(mp=1 << 20, ps=1 << 10), INVALID),
    (dict(plen=-1), INVALID), (dict(plen=5), INVALID), (dict(plen=BIG, pp=P3), INVALID),
    (dict(plen=5, pp=P3 + 1), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=3e38), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(B=1 << 20, H=1 << 12), INVALID),
    (dict(B=1 << 16, H=8, mp=1 << 19, ps=1 << 10), INVALID), (dict(cs=[2048, 1024, 60]), INVALID),
    (dict(cs=[-2048, 1024, 64]), INVALID), (dict(cs=[0, 1024, 64]), INVALID), (dict(cs=[2048, 1024, 0]), INVALID),
])
def test_decode_rejects(kw, status):
    assert _decode(**kw) == status


def test_decode_paged_forwards_its_refusals():
    assert fa.lib().fa_decode_paged(None, P, P, P2, P3, 4, P3, 2, 8, 2, 64, 8, 16, 4, None, 0.125, None, 0, None,
                                    None) == INVALID


def test_workspace_bytes_of_bad_arguments():
    for bad in ((0, 8, 2, 64, 16, 0), (2, 8, 3, 64, 16, 0), (2, 8, 2, 96, 16, 0), (2, 8, 2, 64, 16, -1), (2, 8, 0, 64, 16, 0),
                (2, 8, 2, 64, 0, 5)):
        assert fa.fa_decode_paged_workspace_bytes(*bad) == 0
        assert fa.fa_decode_paged_call_bytes(*bad[:5], 4, *bad[5:]) == 0
    assert fa.fa_decode_paged_call_bytes(2, 8, 2, 64, 16, -1) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    pos, freqs = torch.zeros(8, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        fa.fa_rope(x, x, pos, freqs)
    with pytest.raises(ValueError):
        fa.fa_rope_bwd(x, x, pos, freqs)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_paged_append(x[0].transpose(0, 1), x[0].transpose(0, 1), c, c, torch.zeros(8, dtype=torch.int64))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_decode_paged(q, c, c, table, lens)
    with pytest.raises(ValueError):
        fa.fa_decode_paged_prefix(q, c, c, table[0], 5, table, lens)


def test_rope_freqs():
    f = fa.fa_rope_freqs(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    np.testing.assert_allclose(f.numpy(), [10000.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_and_its_gradient(interleaved):
    """The reference turns each pair as a complex number, its inverse undoes it, and the inverse rotation of an output
    gradient is the gradient: against central differences of a weighted sum."""
    rng = np.random.default_rng(7)
    x = rng.standard_normal((3, 2, 64))
    freqs = 100.0 ** (-np.arange(16) / 16)
    axes = np.arange(16) % 3
    pos = rng.integers(-50, 50, (3, 3))
    y, _ = ref.rotate(x, pos, freqs, axes, interleaved)
    i1, i2 = ref.pairs(32, interleaved)
    phi = np.stack([pos[axes[i]] * freqs[i] for i in range(16)], -1)[:, None]
    z = (x[..., i1] + 1j * x[..., i2]) * np.exp(1j * phi)
    np.testing.assert_allclose(y[..., i1] + 1j * y[..., i2], z, atol=1e-13)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    back, _ = ref.rotate(y, pos, freqs, axes, interleaved, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-13)
    w = rng.standard_normal(x.shape)
    grad, _ = ref.rotate(w, pos, freqs, axes, interleaved, inverse=True)
    h = 1e-5
    for at in [(0, 0, 0), (1, 1, 5), (2, 0, 17), (0, 1, 31), (1, 0, 40)]:
        xp, xm = x.copy(), x.copy()
        xp[at] += h
        xm[at] -= h
        d = ((ref.rotate(xp, pos, freqs, axes, interleaved)[0] - ref.rotate(xm, pos, freqs, axes, interleaved)[0]) * w).sum()
        assert abs(d / (2 * h) - grad[at]) < 1e-8


def test_reference_attention():
    """The reference is the softmax definition, and a sequence's rows come through its pages in order."""
    rng = np.random.default_rng(8)
    q, k, v = rng.standard_normal(64), rng.standard_normal((37, 64)), rng.standard_normal((37, 64))
    o, lse, _, _ = ref.attend(q, k, v, 0.2)
    e = np.exp(0.2 * k @ q)
    np.testing.assert_allclose(o, e @ v / e.sum(), rtol=1e-12)
    assert abs(lse - math.log(e.sum())) < 1e-12
    o, lse, _, _ = ref.attend(q, k[:0], v[:0], 0.2)
    assert (o == 0).all() and lse == -np.inf
    kc, _ = ref.paged_cache(6, 2, 5, 64, "cpu", 9, "one")
    pages, extra, total = ref.deal_pages([11, -1, 0, 5], 5, 10, extra=1)
    assert total == 3 + 0 + 0 + 1 + 1 + 2 and [len(p) for p in pages] == [3, 0, 0, 1] and len(extra) == 1
    kc, vc = ref.paged_cache(total, 2, 5, 64, "cpu", 9, "one")
    rows = ref.sequence_rows(kc, pages[0], 11, 1)
    assert np.array_equal(rows[7], ref.f64(kc[int(pages[0][1]), 1, 2]))
    ref.spoil_unused(kc, vc, pages, [11, -1, 0, 5], extra, 3)
    assert np.isfinite(ref.sequence_rows(kc, pages[0], 11, 1)).all() and torch.isnan(kc).any() and torch.isinf(vc).any()
