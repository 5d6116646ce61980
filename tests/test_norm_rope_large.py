"""The head norms on inputs that give every warp several items one behind the other (its ring's stages are then used again and
again), with the weights' gradients held to a bound that counts the sums as the kernel forms them; and the C entry points with NULL
where the binding always passes something."""
import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref
from paged_ref import f64, rotate

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def draw(shape, dtype, seed, dev, mult=1.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * mult).to(dtype)


def rotation(rot, tokens, dev, n_axes=1):
    freqs = np.array([10000.0 ** (-2 * i / rot) for i in range(rot // 2)])
    axes = np.array([i * n_axes // (rot // 2) for i in range(rot // 2)], dtype=np.int32)
    pos = np.random.default_rng(3).integers(-100, 50_000, (n_axes, *tokens)).astype(np.int32)
    t = lambda x: torch.as_tensor(x, device=dev)  # noqa: E731
    return (pos, freqs, axes), dict(positions=t(pos), freqs=t(freqs), axes=t(axes))


def dw_bound(dy, x, eps, pos, freqs, axes, inter, d, depth):
    """step_ref's bound of dw, but for the sum: each of its terms passes at most `depth` fp32 additions, not all n."""
    g, tg = rotate(dy, pos, freqs, axes, inter, inverse=True)
    u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    rest = tuple(range(x.ndim - 1))
    e = (d / 2 + 4) * ref.U32 + 2.0 ** -22
    terms = np.abs(g * u)
    return (tg * np.abs(u) + (e + 2 * ref.U32) * terms).sum(rest) + depth * ref.U32 * terms.sum(rest)


# B, H, Hkv, N, d, dtype, interleaved, rot
LARGE = [(2, 12, 2, 4097, 128, BF, False, 128), (1, 8, 8, 6001, 64, F32, True, 32), (3, 3, 1, 9001, 64, BF, False, 64)]


@pytest.mark.parametrize("case", LARGE)
def test_forward_and_backward(cuda_device, case):
    B, H, Hkv, N, d, dt, inter, rot = case
    whole = draw((B, N, H + Hkv + 1, d), dt, 1, cuda_device, 2.0)
    q, k = whole[:, :, :H].transpose(1, 2), whole[:, :, H:H + Hkv].transpose(1, 2)
    wq, wk = draw((d,), dt, 4, cuda_device), draw((d,), F32 if dt == F32 else BF, 5, cuda_device)
    dq, dk = draw((B, H, N, d), dt, 7, cuda_device), draw((B, Hkv, N, d), dt, 8, cuda_device)
    turn, how = rotation(rot, (B, N), cuda_device)
    qo, ko = fa.fa_norm_rope(q, k, wq, wk, interleaved=inter, eps=EPS, **how)
    out = fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, interleaved=inter, eps=EPS, **how)
    assert fa.fa_check_device_error() == fa.FA_OK
    # A lane adds at most 16 heads' terms an item; a warp has at most ceil(items / warps) of a kind's items, where all warps of three
    # blocks an SM take part once there are as many items, of a token each at least.  Then 2 to 5 lanes' sums, 4 warps', and the
    # blocks' shares, an eighth of them in turn and the 8 sums.
    warps = torch.cuda.get_device_properties(cuda_device).multi_processor_count * 3 * 4
    depth = 16 * -(-B * N // warps) + 5 + 4 + warps // 4 // 8 + 1 + 8
    assert depth < B * N * Hkv / 16  # far below the number of terms
    for y, gx, gw, dy, x, w, name in ((qo, out[0], out[2], dq, q, wq, "q"), (ko, out[1], out[3], dk, k, wk, "k")):
        x64, dy64 = f64(x.transpose(1, 2)), f64(dy.transpose(1, 2))
        ref.check(y.transpose(1, 2), *ref.norm_rope(x64, f64(w), EPS, *turn, inter), name)
        dx, dw, tol, _ = ref.norm_rope_bwd(dy64, x64, f64(w), EPS, *turn, inter)
        ref.check(gx.transpose(1, 2), dx, tol, "d" + name)
        ref.check(gw, dw, dw_bound(dy64, x64, EPS, *turn, inter, d, depth), f"d{name}_weight")


@pytest.mark.parametrize("H,Hkv,d,rot,inter,T,ps", [(8, 2, 128, 128, False, 12_001, 16), (4, 4, 64, 32, True, 9_999, 24), (0, 2, 128, 64, False, 9_001, 7)])
def test_append_of_a_prompt(cuda_device, H, Hkv, d, rot, inter, T, ps):
    pages = -(-T // ps) + 5
    kc, vc = draw((pages, Hkv, ps, d), BF, 1, cuda_device), draw((pages, Hkv, ps, d), BF, 9, cuda_device)
    kc0, vc0 = kc.clone(), vc.clone()
    whole = draw((T, H + 2 * Hkv, d), BF, 2, cuda_device, 3.0)
    q, k, v = whole[:, :H] if H else None, whole[:, H:H + Hkv], whole[:, H + Hkv:]
    wq, wk = draw((d,), BF, 4, cuda_device) if H else None, draw((d,), BF, 5, cuda_device)
    slots = np.random.default_rng(T).permutation(pages * ps)[:T]
    slots[T - 300:T - 100] = -1  # places without a token, and tokens behind them
    stored = slots >= 0
    turn, how = rotation(rot, (T,), cuda_device)
    got = fa.fa_paged_append(k, v, kc, vc, torch.as_tensor(slots, device=cuda_device), q=q, interleaved=inter, q_weight=wq, k_weight=wk,
                             eps=EPS, **how)
    assert fa.fa_check_device_error() == fa.FA_OK
    if H:
        ref.check(got, *ref.norm_rope(f64(q), f64(wq), EPS, *turn, inter), "q")
    y, tol = ref.norm_rope(f64(k), f64(wk), EPS, *turn, inter)
    page, row = (torch.as_tensor(x, device=cuda_device) for x in (slots[stored] // ps, slots[stored] % ps))
    ref.check(kc[page, :, row], y[stored], tol[stored], "keys")
    assert torch.equal(vc[page, :, row], v[torch.as_tensor(stored, device=cuda_device)])
    kc0[page, :, row], vc0[page, :, row] = kc[page, :, row], vc[page, :, row]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)  # nothing else changed


@pytest.mark.parametrize("dtype", [BF, F32])
def test_c_entry_points_with_null(cuda_device, dtype):
    """NULL strides (all contiguous) and a NULL workspace, eager, on another stream and captured: the binding's results."""
    B, H, Hkv, N, d, ps = 2, 6, 2, 77, 64, 16
    L, ty = fa.lib(), fa.FA_BF16 if dtype == BF else fa.FA_FP32
    q, k, dq, dk = (draw((B, h, N, d), dtype, i, cuda_device) for i, h in enumerate((H, Hkv, H, Hkv)))
    wq, wk = draw((d,), dtype, 4, cuda_device), draw((d,), dtype, 5, cuda_device)
    _, how = rotation(d, (B, N), cuda_device)
    want = fa.fa_norm_rope(q, k, wq, wk, eps=EPS, **how)
    grads = fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, eps=EPS, **how)
    torch.cuda.synchronize()
    outs = [torch.empty_like(t) for t in (*want, *grads)]
    p = lambda *ts: [t.data_ptr() for t in ts]  # noqa: E731
    tail = (*p(wq, wk), ty, EPS, *p(how["positions"]), 0, *p(how["freqs"], how["axes"]), 1, d, 0)

    def forward(stream):
        return L.fa_norm_rope(*p(q, k, *outs[:2]), None, B, H, Hkv, N, d, ty, *tail, stream.cuda_stream)

    def backward(stream):
        return L.fa_norm_rope_bwd(*p(dq, dk, q, k, *outs[2:]), None, B, H, Hkv, N, d, ty, *tail, None, 0, stream.cuda_stream)

    def check():
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_OK
        for got, right in zip(outs, (*want, *grads)):
            assert torch.equal(got, right)
            got.fill_(float("nan"))
        torch.cuda.synchronize()

    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        assert forward(stream) == fa.FA_OK and backward(stream) == fa.FA_OK
        check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        assert forward(torch.cuda.current_stream()) == fa.FA_OK and backward(torch.cuda.current_stream()) == fa.FA_OK
    for _ in range(2):
        graph.replay()
        check()
    if dtype == BF:  # the append: contiguous tokens and caches
        T = N
        kt, vt, qt = (draw((T, h, d), BF, 11 + h, cuda_device) for h in (Hkv, Hkv, H))
        slots = torch.randperm(6 * ps, device=cuda_device)[:T].contiguous()
        turn = dict(positions=how["positions"][:, 0].contiguous(), freqs=how["freqs"], axes=how["axes"])
        caches = [[torch.zeros(6, Hkv, ps, d, dtype=BF, device=cuda_device) for _ in range(2)] for _ in range(2)]
        right = fa.fa_paged_append(kt, vt, *caches[0], slots, q=qt, q_weight=wq, k_weight=wk, eps=EPS, **turn)
        got = torch.empty_like(qt)
        st = L.fa_paged_append_norm(*p(kt, vt, qt, got, *caches[1]), None, None, *p(slots), T, H, Hkv, d, 6, ps, *p(wq, wk), ty, EPS,
                                    *p(turn["positions"], turn["freqs"], turn["axes"]), 1, d, 0, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == fa.FA_OK and torch.equal(got, right)
        assert all(torch.equal(a, b) for a, b in zip(*caches))
