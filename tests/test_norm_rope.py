"""fa_norm_rope, fa_norm_rope_bwd and the normed fa_paged_append against their float64 definitions."""
import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref
from paged_ref import f64, paged_cache

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def draw(shape, dtype, seed, dev, mult=1.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * mult).to(dtype)


def rotation(rot, n_axes, tokens, dev, seed=3, far=50_000):
    rng = np.random.default_rng(seed)
    freqs = np.array([10000.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)])
    axes = np.array([i * n_axes // max(1, rot // 2) for i in range(rot // 2)], dtype=np.int32)
    pos = rng.integers(-100, far, (n_axes, *tokens)).astype(np.int32)
    t = lambda x: torch.as_tensor(x, device=dev)  # noqa: E731
    return (freqs, axes, pos), dict(positions=t(pos), freqs=t(freqs)), t(axes)


# B, H, Hkv, N, d, dtype, weights' dtype, axes, interleaved, rot
CASES = [
    (1, 1, 0, 1, 64, BF, BF, 1, False, 64), (1, 1, 1, 1, 128, BF, F32, 1, False, 128), (2, 2, 1, 37, 64, F32, F32, 1, False, 64),
    (1, 3, 1, 65, 128, F32, F32, 3, True, 128), (2, 8, 2, 33, 64, BF, BF, 1, False, 32), (1, 5, 5, 17, 128, BF, F32, 3, True, 48),
    (3, 12, 3, 9, 64, BF, BF, 2, True, 64), (1, 16, 4, 333, 64, F32, F32, 3, False, 64), (1, 40, 8, 5, 128, BF, BF, 1, False, 128),
    (1, 4, 2, 11, 128, F32, BF, 1, False, 16), (2, 32, 8, 129, 128, BF, BF, 1, False, 128), (1, 7, 1, 300, 64, BF, BF, 1, True, 16),
]


def inputs(case, dev, layout):
    B, H, Hkv, N, d, dt, wt, n_axes, inter, rot = case
    if layout == "projection":  # heads of one projection's output [B, N, heads, d], padded
        whole = draw((B, N, H + Hkv + 1, d), dt, 1, dev, 2.0)
        q, k = whole[:, :, :H].transpose(1, 2), whole[:, :, H:H + Hkv].transpose(1, 2) if Hkv else None
    else:
        q, k = draw((B, H, N, d), dt, 1, dev, 2.0), draw((B, Hkv, N, d), dt, 2, dev, 2.0) if Hkv else None
    if N > 3:
        q[0, 0, 2] = 0  # a head of zeros: eps alone
        q[0, 0, 3] *= 2.0 ** -20
    wq, wk = draw((d,), wt, 4, dev), draw((d,), wt, 5, dev) if Hkv else None
    return q, k, wq, wk


@pytest.mark.parametrize("layout", ["dense", "projection"])
@pytest.mark.parametrize("case", CASES)
def test_forward(cuda_device, case, layout):
    B, H, Hkv, N, d, dt, wt, n_axes, inter, rot = case
    q, k, wq, wk = inputs(case, cuda_device, layout)
    (freqs, axes, pos), how, ax = rotation(rot, n_axes, (B, N), cuda_device)
    qo, ko = fa.fa_norm_rope(q, k, wq, wk, axes=ax, interleaved=inter, eps=EPS, **how)
    assert qo.is_contiguous() and (ko is None) == (k is None)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        if x is not None:
            y, tol = ref.norm_rope(f64(x.transpose(1, 2)), f64(w), EPS, pos, freqs, axes, inter)
            ref.check(got.transpose(1, 2), y, tol, "norm_rope")
    assert fa.fa_check_device_error() == fa.FA_OK


@pytest.mark.parametrize("layout", ["dense", "projection"])
@pytest.mark.parametrize("case", CASES)
def test_backward(cuda_device, case, layout):
    B, H, Hkv, N, d, dt, wt, n_axes, inter, rot = case
    q, k, wq, wk = inputs(case, cuda_device, layout)
    dq = draw((B, H, N, d), dt, 7, cuda_device)
    dk = draw((B, Hkv, N, d), dt, 8, cuda_device) if Hkv else None
    (freqs, axes, pos), how, ax = rotation(rot, n_axes, (B, N), cuda_device)
    out = fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, axes=ax, interleaved=inter, eps=EPS, **how)
    for gx, gw, dy, x, w in ((out[0], out[2], dq, q, wq), (out[1], out[3], dk, k, wk)):
        if x is None:
            assert gx is None and gw is None
            continue
        dx, dw, tol, tol_w = ref.norm_rope_bwd(f64(dy.transpose(1, 2)), f64(x.transpose(1, 2)), f64(w), EPS, pos, freqs, axes,
                                               inter)
        ref.check(gx.transpose(1, 2), dx, tol, "dx")
        assert gw.dtype == F32
        ref.check(gw, dw, tol_w, "dw")


@pytest.mark.parametrize("d,dt", [(64, BF), (128, F32)])
def test_without_rotation(cuda_device, d, dt):
    case = (2, 6, 2, 21, d, dt, dt, 1, False, 0)
    q, k, wq, wk = inputs(case, cuda_device, "dense")
    qo, ko = fa.fa_norm_rope(q, k, wq, wk, None, None, eps=EPS)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        ref.check(got, *ref.norm_rope(f64(x), f64(w), EPS), "norm")
    dq, dk = draw(q.shape, dt, 7, cuda_device), draw(k.shape, dt, 8, cuda_device)
    a, b, c, e = fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, None, None, eps=EPS)
    for gx, gw, dy, x, w in ((a, c, dq, q, wq), (b, e, dk, k, wk)):
        dx, dw, tol, tol_w = ref.norm_rope_bwd(f64(dy), f64(x), f64(w), EPS)
        ref.check(gx, dx, tol, "dx")
        ref.check(gw, dw, tol_w, "dw")


def test_gradient_against_differences(cuda_device):
    """The kernels' own forward pass on both sides of a small step, fp32.  The step h leaves the formula's remainder, taken from
    the float64 reference; the outputs' roundings leave at most sum |dy| bound(y) / h."""
    case = (1, 3, 2, 19, 64, F32, F32, 1, False, 64)
    q, k, wq, wk = inputs(case, cuda_device, "dense")
    q[0, 0, 2:4] = 1.0  # far from the norm's corner at zero
    (freqs, axes, pos), how, ax = rotation(64, 1, (1, 19), cuda_device)
    dq, dk = draw(q.shape, F32, 7, cuda_device), draw(k.shape, F32, 8, cuda_device)
    out = fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, axes=ax, eps=EPS, **how)
    h = 2.0 ** -7
    steps = [draw(x.shape, F32, 20 + i, cuda_device) for i, x in enumerate((q, k, wq, wk))]
    sides, exact, slack = [], [], 0.0
    for sign in (1, -1):
        xs = [x + sign * h * s for x, s in zip((q, k, wq, wk), steps)]
        qo, ko = fa.fa_norm_rope(*xs, axes=ax, eps=EPS, **how)
        sides.append(float((qo.double() * dq).sum() + (ko.double() * dk).sum()))
        total = 0.0
        for x, w, dy in ((xs[0], xs[2], dq), (xs[1], xs[3], dk)):
            y, tol = ref.norm_rope(f64(x.transpose(1, 2)), f64(w), EPS, pos, freqs, axes)
            g = f64(dy.transpose(1, 2))
            total += (y * g).sum()
            slack += (np.abs(g) * (tol + ref.U32 * np.abs(y))).sum() / (2 * h)
        exact.append(total)
    along = sum(float((g.double() * s).sum()) for g, s in zip(out, steps))
    # the float64 difference and the float64 derivative, for the remainder
    true = 0.0
    for x, w, dy, sx, sw in ((q, wq, dq, steps[0], steps[2]), (k, wk, dk, steps[1], steps[3])):
        dx, dw, tol, tol_w = ref.norm_rope_bwd(f64(dy.transpose(1, 2)), f64(x.transpose(1, 2)), f64(w), EPS, pos, freqs, axes)
        true += (dx * f64(sx.transpose(1, 2))).sum() + (dw * f64(sw)).sum()
        slack += ((tol + ref.U32 * np.abs(dx)) * np.abs(f64(sx.transpose(1, 2)))).sum()
        slack += ((tol_w + ref.U32 * np.abs(dw)) * np.abs(f64(sw))).sum()
    remainder = abs((exact[0] - exact[1]) / (2 * h) - true)
    assert remainder < 0.05 * abs(true)  # the step is small enough to say something
    assert abs((sides[0] - sides[1]) / (2 * h) - along) <= remainder + slack


def test_in_place(cuda_device):
    case = (2, 8, 2, 33, 64, BF, BF, 1, False, 64)
    q, k, wq, wk = inputs(case, cuda_device, "projection")
    _, how, ax = rotation(64, 1, (2, 33), cuda_device)
    want = fa.fa_norm_rope(q, k, wq, wk, axes=ax, eps=EPS, **how)
    dq, dk = draw(q.shape, BF, 7, cuda_device), draw(k.shape, BF, 8, cuda_device)
    grads = fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, axes=ax, eps=EPS, **how)
    for over in ("gradient", "input"):
        a, b, x, y = dq.clone(), dk.clone(), q.clone(), k.clone()
        ins = (a, b) if over == "gradient" else (x, y)
        got = fa.fa_norm_rope_bwd(a, b, x, y, wq, wk, axes=ax, eps=EPS, dq_in=ins[0], dk_in=ins[1], **how)
        assert got[0] is ins[0] and got[1] is ins[1]
        assert all(torch.equal(g, w) for g, w in zip(got, grads))
    got = fa.fa_norm_rope(q, k, wq, wk, axes=ax, eps=EPS, q_out=q, k_out=k, **how)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_backward_is_reproducible_on_streams_and_in_graphs(cuda_device):
    """Many tokens; the same bits from eager calls, another stream and two captured graphs with a workspace each."""
    case = (2, 16, 4, 2500, 128, BF, BF, 1, False, 128)
    q, k, wq, wk = inputs(case, cuda_device, "dense")
    _, how, ax = rotation(128, 1, (2, 2500), cuda_device)
    dq, dk = draw(q.shape, BF, 7, cuda_device), draw(k.shape, BF, 8, cuda_device)

    def go(**kw):
        return fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, axes=ax, eps=EPS, **how, **kw)

    want = go()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = go(stream=s)
    s.synchronize()
    graphs = []
    for _ in range(2):
        ws = torch.empty(fa.fa_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8, device=cuda_device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = go(workspace=ws)
        graphs.append((g, out, ws))
    for _ in range(3):
        for g, _, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for got in (other, graphs[0][1], graphs[1][1]):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and the sums over 5000 tokens' heads
    B, N = 2, 2500
    x, dy = f64(k.transpose(1, 2)), f64(dk.transpose(1, 2))
    freqs, pos = f64(how["freqs"]), how["positions"].cpu().numpy()
    dx, dw, tol, tol_w = ref.norm_rope_bwd(dy, x, f64(wk), EPS, pos, freqs, ax.cpu().numpy())
    ref.check(want[1].transpose(1, 2), dx, tol, "dk")
    ref.check(want[3], dw, tol_w, "dk_weight")


def test_axis_out_of_range_is_reported(cuda_device):
    case = (1, 4, 2, 8, 64, BF, BF, 1, False, 64)
    q, k, wq, wk = inputs(case, cuda_device, "dense")
    _, how, ax = rotation(64, 1, (1, 8), cuda_device)
    ax[5] = 1
    qo, _ = fa.fa_norm_rope(q, k, wq, wk, axes=ax, eps=EPS, **how)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG
    bad = torch.isnan(qo)
    assert bad[..., [5, 37]].all() and bad.sum() == 2 * qo.shape[1] * qo.shape[2]


def test_no_tokens(cuda_device):
    x, w = torch.empty(2, 4, 0, 64, dtype=BF, device=cuda_device), draw((64,), BF, 1, cuda_device)
    pos, freqs = torch.empty(0, dtype=torch.int32, device=cuda_device), fa.fa_rope_freqs(64)
    assert fa.fa_norm_rope(x, x, w, w, pos, freqs)[0].shape == x.shape
    out = fa.fa_norm_rope_bwd(x, x, x, x, w, w, pos, freqs)
    assert out[0].shape == x.shape and not out[2].any() and not out[3].any()


@pytest.mark.parametrize("H,Hkv,d,rot,inter,n_axes,layout", [
    (8, 2, 64, 64, False, 1, "head"), (32, 8, 128, 128, True, 3, "row"), (4, 4, 64, 32, False, 1, "one"), (0, 2, 128, 128, False, 1, "odd"),
    (6, 1, 128, 0, False, 1, "head"),
])
@pytest.mark.parametrize("T", [1, 50])
def test_append(cuda_device, H, Hkv, d, rot, inter, n_axes, layout, T):
    ps = 16
    kc, vc = paged_cache(8, Hkv, ps, d, cuda_device, 1, layout)
    kc0, vc0 = f64(kc), f64(vc)
    whole = draw((T, H + 2 * Hkv, d), BF, 2, cuda_device, 3.0)
    q, k, v = whole[:, :H] if H else None, whole[:, H:H + Hkv], whole[:, H + Hkv:]
    wq, wk = draw((d,), F32, 4, cuda_device) if H else None, draw((d,), F32, 5, cuda_device)
    rng = np.random.default_rng(T)
    slots = rng.permutation(8 * ps)[:T]
    slots[T // 2:T // 2 + 3] = -1
    (freqs, axes, pos), how, ax = rotation(rot, n_axes, (T,), cuda_device)
    if not rot:
        how, ax = dict(positions=None, freqs=None), None
    got = fa.fa_paged_append(k, v, kc, vc, torch.as_tensor(slots, device=cuda_device), q=q, axes=ax, interleaved=inter,
                             q_weight=wq, k_weight=wk, eps=EPS, **how)
    rotated = (pos, freqs, axes, inter) if rot else ()
    if H:
        ref.check(got, *ref.norm_rope(f64(q), f64(wq), EPS, *rotated), "q")
    y, tol = ref.norm_rope(f64(k), f64(wk), EPS, *rotated)
    want_k, tol_k, want_v = kc0.copy(), np.zeros_like(kc0), vc0.copy()
    for t, s in enumerate(slots):
        if s >= 0:
            want_k[s // ps, :, s % ps], tol_k[s // ps, :, s % ps], want_v[s // ps, :, s % ps] = y[t], tol[t], f64(v)[t]
    untouched = tol_k == 0
    assert np.array_equal(f64(kc)[untouched], want_k[untouched]) and np.array_equal(f64(vc), want_v)
    ref.check(kc, want_k, tol_k, "k_cache")
    assert fa.fa_check_device_error() == fa.FA_OK
