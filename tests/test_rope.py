"""GPU parity of fa_rope, fa_rope_bwd and fa_paged_append against the float64 references (tests/paged_ref.py), within
bounds counted from the kernels' roundings."""
import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import paged_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _draw(shape, seed, dev, dtype=torch.bfloat16):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(dtype)


def _rotation(rot, n_axes, dev, seed, theta=10000.0):
    freqs = fa.fa_rope_freqs(rot, theta, device=dev)
    axes = np.random.default_rng(seed).integers(0, n_axes, rot // 2).astype(np.int32)
    return freqs, torch.as_tensor(axes, device=dev), axes


def _check_rope(q, k, qo, ko, pos, freqs, axes, inter, inverse, name):
    """pos: numpy [A, B, N].  Rows of heads are [B, N, heads, d]."""
    for n, x, y in (("q", q, qo), ("k", k, ko)):
        if x is None:
            assert y is None
            continue
        r, tol = ref.rotate(ref.f64(x.transpose(1, 2)), pos, ref.f64(freqs), axes, inter, inverse)
        ref.check_rotated(y.transpose(1, 2), r, tol, f"{name} {n}")


def _ok():
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48)])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 5, 1, 33), (3, 4, 2, 257)], ids=str)
def test_rope_forward_and_backward(cuda_device, dtype, d, rot, inter, shape):
    B, H, Hkv, N = shape
    n_axes = 1 + N % 3
    q, k = _draw((B, H, N, d), 1, cuda_device, DT[dtype]), _draw((B, Hkv, N, d), 2, cuda_device, DT[dtype])
    freqs, axes_t, axes = _rotation(rot, n_axes, cuda_device, 3)
    pos = np.random.default_rng(4).integers(-1000, 200_000, (n_axes, B, N)).astype(np.int32)
    pos_t = torch.as_tensor(pos, device=cuda_device)
    q0, k0 = q.clone(), k.clone()
    for inverse, call in ((False, fa.fa_rope), (True, fa.fa_rope_bwd)):
        qo, ko = call(q, k, pos_t, freqs, axes=axes_t, interleaved=inter)
        _ok()
        assert torch.equal(q, q0) and torch.equal(k, k0)
        _check_rope(q, k, qo, ko, pos, freqs, axes, inter, inverse, f"rope {dtype} d{d} rot{rot} {shape}")


def test_rope_backward_is_the_gradient(cuda_device):
    """Central differences of a weighted sum of fa_rope's fp32 outputs against fa_rope_bwd of the weights.  The map is
    linear, so the difference quotient is exact but for fp32 rounding: |y| u / h with h = 1 in each direction."""
    B, H, N, d = 1, 2, 9, 64
    q = _draw((B, H, N, d), 11, cuda_device, torch.float32)
    w = _draw((B, H, N, d), 12, cuda_device, torch.float32)
    freqs, axes_t, _ = _rotation(64, 3, cuda_device, 13, theta=30.0)
    pos = torch.as_tensor(np.random.default_rng(14).integers(0, 99, (3, B, N)).astype(np.int32), device=cuda_device)
    grad, _ = fa.fa_rope_bwd(w, None, pos, freqs, axes=axes_t)
    for at in [(0, 0, 0, 0), (0, 1, 4, 31), (0, 0, 8, 32), (0, 1, 3, 63)]:
        up, down = q.clone(), q.clone()
        up[at] += 1.0
        down[at] -= 1.0
        diff = fa.fa_rope(up, None, pos, freqs, axes=axes_t)[0].double() - fa.fa_rope(down, None, pos, freqs, axes=axes_t)[0].double()
        fd = (diff * w.double()).sum().item() / 2
        # two outputs change; each is off by 4.5e-7 (|x1| + |x2|) with |x| <= 6, weights below 5
        assert abs(fd - grad[at].item()) <= 2 * 2 * 5 * 4.5e-7 * 12
    _ok()


@pytest.mark.parametrize("value", [0, 1, -1, 999_999_937, -2 ** 31, 2 ** 31 - 1])
def test_rope_far_positions(cuda_device, value):
    q = _draw((1, 2, 4, 128), 21, cuda_device, torch.float32)
    freqs = fa.fa_rope_freqs(128, device=cuda_device)
    pos = torch.full((4,), value, dtype=torch.int32, device=cuda_device)
    qo, _ = fa.fa_rope(q, None, pos, freqs)
    _ok()
    _check_rope(q, None, qo, None, np.full((1, 1, 4), value, np.int32), freqs, np.zeros(64, int), False, False, f"far {value}")
    if value == 0:
        assert torch.equal(qo, q)


def test_rope_odd_frequencies(cuda_device):
    """Frequencies above a turn a position, negative ones and zero."""
    freqs = torch.tensor([0.0, -0.3, 7.5, 2 * np.pi, -100.25, 1e-9, 3.0, 1.0], dtype=torch.float64, device=cuda_device)
    q = _draw((2, 3, 17, 64), 22, cuda_device, torch.float32)
    pos = np.random.default_rng(23).integers(-5000, 5000, (1, 1, 17)).astype(np.int32)
    qo, _ = fa.fa_rope(q, None, torch.as_tensor(pos[0, 0], device=cuda_device), freqs)
    _ok()
    _check_rope(q, None, qo, None, np.broadcast_to(pos, (1, 2, 17)), freqs, np.zeros(8, int), False, False, "odd freqs")


def test_rope_strided_inputs_in_place_and_shared_positions(cuda_device):
    """Heads read out of one projection's [B, N, heads, d] output; rotated in place there; positions [A, 1, N]."""
    B, N, H, Hkv, d = 2, 75, 6, 2, 64
    x = _draw((B, N, H + 2 * Hkv, d), 31, cuda_device)
    x0 = x.clone()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    freqs, axes_t, axes = _rotation(32, 2, cuda_device, 32)
    pos = np.random.default_rng(33).integers(0, 5000, (2, 1, N)).astype(np.int32)
    pos_t = torch.as_tensor(pos, device=cuda_device)
    full = np.broadcast_to(pos, (2, B, N))
    qo, ko = fa.fa_rope(q, k, pos_t, freqs, axes=axes_t)
    _ok()
    assert qo.is_contiguous() and ko.is_contiguous() and torch.equal(x, x0)
    _check_rope(q, k, qo, ko, full, freqs, axes, False, False, "strided")
    a, b = fa.fa_rope(q, k, pos_t, freqs, axes=axes_t, q_out=q, k_out=k)
    _ok()
    assert a is q and b is k and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, :, H + Hkv:], x0[:, :, H + Hkv:])


def test_rope_many_heads_and_tokens(cuda_device):
    """More heads than one thread walks, enough tokens to fill the GPU, odd counts of both; sampled tokens."""
    B, H, Hkv, N, d = 3, 37, 11, 4099, 128
    q, k = _draw((B, H, N, d), 41, cuda_device), _draw((B, Hkv, N, d), 42, cuda_device)
    freqs, axes_t, axes = _rotation(128, 3, cuda_device, 43)
    pos = np.random.default_rng(44).integers(0, 1 << 20, (3, B, N)).astype(np.int32)
    qo, ko = fa.fa_rope(q, k, torch.as_tensor(pos, device=cuda_device), freqs, axes=axes_t)
    _ok()
    at = sorted({0, 1, 31, 32, N - 1, *np.random.default_rng(45).integers(0, N, 40).tolist()})
    idx = torch.as_tensor(at, device=cuda_device)
    _check_rope(q[:, :, idx], k[:, :, idx], qo[:, :, idx], ko[:, :, idx], pos[:, :, at], freqs, axes, False, False, "many")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv,N,d,rot,inter", [
    (1, 0, 41_003, 64, 64, False), (2, 0, 21_001, 128, 128, True), (2, 1, 30_001, 64, 32, True), (1, 1, 25_002, 128, 112, False),
    (4, 0, 33_333, 64, 64, True), (40, 5, 3001, 64, 48, False)], ids=str)
def test_rope_tokens_in_many_rounds(cuda_device, dtype, H, Hkv, N, d, rot, inter):
    """Every warp takes several items; few heads and more; outputs in place."""
    q = _draw((1, H, N, d), 46, cuda_device, DT[dtype])
    k = _draw((1, Hkv, N, d), 47, cuda_device, DT[dtype]) if Hkv else None
    freqs, axes_t, axes = _rotation(rot, 8, cuda_device, 48)
    pos = np.random.default_rng(49).integers(-(1 << 16), 1 << 16, (8, 1, N)).astype(np.int32)
    qo, ko = q.clone(), None if k is None else k.clone()
    fa.fa_rope(qo, ko, torch.as_tensor(pos, device=cuda_device), freqs, axes=axes_t, interleaved=inter, q_out=qo, k_out=ko)
    _ok()
    at = sorted({0, 1, 7, 8, N - 2, N - 1, *np.random.default_rng(50).integers(0, N, 300).tolist()})
    idx = torch.as_tensor(at, device=cuda_device)
    _check_rope(q[:, :, idx], None if k is None else k[:, :, idx], qo[:, :, idx], None if ko is None else ko[:, :, idx],
                pos[:, :, at], freqs, axes, inter, False, f"rounds {dtype} H{H}/{Hkv} d{d}")


def test_rope_bad_axis_is_nan_and_reported(cuda_device):
    q = _draw((1, 2, 5, 64), 51, cuda_device, torch.float32)
    freqs = fa.fa_rope_freqs(64, device=cuda_device)
    axes = torch.zeros(32, dtype=torch.int32, device=cuda_device)
    axes[3], axes[9] = 2, -1
    pos = torch.arange(5, dtype=torch.int32, device=cuda_device)
    qo, _ = fa.fa_rope(q, None, pos, freqs, axes=axes)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG
    assert fa.fa_check_device_error() == fa.FA_OK
    bad = torch.zeros(64, dtype=torch.bool, device=cuda_device)
    bad[[3, 35, 9, 41]] = True
    assert torch.equal(torch.isnan(qo), bad.expand_as(qo))


def test_rope_refusals(cuda_device):
    q = _draw((2, 2, 5, 64), 52, cuda_device)
    freqs = fa.fa_rope_freqs(64, device=cuda_device)
    pos = torch.arange(5, dtype=torch.int32, device=cuda_device)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:4]), dict(freqs=freqs.float()), dict(k=q.float()),
                dict(k=q[:, :, :4]), dict(axes=torch.zeros(31, dtype=torch.int32, device=cuda_device)),
                dict(q=q.transpose(2, 3)), dict(q_out=q.float()), dict(q=q.to(torch.float16)),
                dict(freqs=freqs.cpu()), dict(k_out=q)):
        a = dict(q=q, k=None, positions=pos, freqs=freqs)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            fa.fa_rope(**a)
    with pytest.raises(fa.FAError):  # 8-byte aligned rows
        fa.fa_rope(torch.empty(2, 2, 5, 68, device=cuda_device, dtype=torch.bfloat16)[..., :64], None, pos, freqs)
    _ok()


# ------------------------------------------------------------------------------------------ append

def _append_case(dev, T, H, Hkv, d, ps, layout, seed, negative=0.2):
    rng = np.random.default_rng(seed)
    pages = -(-T // ps) + 3
    kc, vc = ref.paged_cache(pages, Hkv, ps, d, dev, seed, layout)
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    slots[rng.random(T) < negative] = -1 - rng.integers(0, 3)
    x = _draw((T, H + 2 * Hkv, d), seed + 1, dev)
    return kc, vc, slots, x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


def _check_append(kc0, vc0, kc, vc, slots, k, v, rk, tk, ps, name):
    """Every named row holds the token's (rotated) key and value; every other row is as it was, bit for bit."""
    want_v = vc0.clone()
    seen = torch.zeros(kc.shape[0], ps, dtype=torch.bool)
    for t, s in enumerate(slots):
        if s >= 0:
            want_v[int(s) // ps, :, int(s) % ps] = v[t]
            seen[int(s) // ps, int(s) % ps] = True
            ref.check_rotated(kc[int(s) // ps, :, int(s) % ps], rk[t], tk[t], f"{name} token {t}")
    assert torch.equal(vc, want_v), name
    free = (~seen).to(kc.device)[:, None, :, None].expand(kc.shape)
    assert torch.equal(kc[free], kc0[free]), name


@pytest.mark.parametrize("layout", ["head", "row", "one", "odd"])
@pytest.mark.parametrize("d,rot,inter,ps", [(64, 64, False, 16), (128, 32, True, 1), (128, 128, False, 24), (64, 0, False, 100)])
@pytest.mark.parametrize("T,H,Hkv", [(1, 8, 2), (37, 0, 3), (300, 5, 5)])
def test_append(cuda_device, layout, d, rot, inter, ps, T, H, Hkv):
    kc, vc, slots, q, k, v = _append_case(cuda_device, T, H, Hkv, d, ps, layout, 100 + T + d + ps)
    if T == 1:
        slots[0] = 2 * ps
    kc0, vc0 = kc.clone(), vc.clone()
    n_axes = 2
    kw, axes, pos = {}, None, np.random.default_rng(5).integers(-9, 90_000, (n_axes, T)).astype(np.int32)
    if rot:
        freqs, axes_t, axes = _rotation(rot, n_axes, cuda_device, 6)
        kw = dict(positions=torch.as_tensor(pos, device=cuda_device), freqs=freqs, axes=axes_t, interleaved=inter)
    qo = fa.fa_paged_append(k, v, kc, vc, torch.as_tensor(slots, device=cuda_device), q=q if H else None, **kw)
    _ok()
    name = f"append {layout} d{d} rot{rot} ps{ps} T{T}"
    fr = ref.f64(kw["freqs"]) if rot else np.zeros(0)
    rk, tk = ref.rotate(ref.f64(k), pos, fr, axes, inter)
    _check_append(kc0, vc0, kc, vc, slots, k, v, rk, tk, ps, name)
    if H:
        rq, tq = ref.rotate(ref.f64(q), pos, fr, axes, inter)
        ref.check_rotated(qo, rq, tq, name + " q")
    else:
        assert qo is None


def test_append_long_prompt(cuda_device):
    """Enough tokens that a thread walks several heads; one axis as a plain vector."""
    T, H, Hkv, d, ps = 4097, 33, 3, 64, 64
    kc, vc, slots, q, k, v = _append_case(cuda_device, T, H, Hkv, d, ps, "head", 200, negative=0.01)
    kc0, vc0 = kc.clone(), vc.clone()
    freqs = fa.fa_rope_freqs(d, device=cuda_device)
    pos = np.arange(T, dtype=np.int32) + 100_000
    qo = fa.fa_paged_append(k, v, kc, vc, torch.as_tensor(slots, device=cuda_device), q=q,
                            positions=torch.as_tensor(pos, device=cuda_device), freqs=freqs)
    _ok()
    rk, tk = ref.rotate(ref.f64(k), pos[None], ref.f64(freqs), np.zeros(32, int), False)
    _check_append(kc0, vc0, kc, vc, slots, k, v, rk, tk, ps, "append long")
    rq, tq = ref.rotate(ref.f64(q), pos[None], ref.f64(freqs), np.zeros(32, int), False)
    ref.check_rotated(qo, rq, tq, "append long q")


def test_append_in_place_queries_and_no_tokens(cuda_device):
    kc, vc, slots, _, k, v = _append_case(cuda_device, 19, 4, 2, 64, 16, "head", 300)
    q = _draw((19, 4, 64), 301, cuda_device)
    freqs = fa.fa_rope_freqs(64, device=cuda_device)
    pos = torch.arange(19, dtype=torch.int32, device=cuda_device)
    st = torch.as_tensor(slots, device=cuda_device)
    a = fa.fa_paged_append(k, v, kc, vc, st, q=q.clone(), positions=pos, freqs=freqs)
    b = fa.fa_paged_append(k, v, kc, vc, st, q=q, positions=pos, freqs=freqs, q_out=q)
    assert b is q and torch.equal(a, q)
    before = kc.clone()
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    assert fa.fa_paged_append(e, e, kc, vc, st[:0]) is None
    _ok()
    assert torch.equal(kc, before)


def test_append_slot_past_the_cache_is_reported(cuda_device):
    """A slot at or past num_pages * page_size stores nothing and is reported; the other tokens are stored."""
    kc, vc, slots, q, k, v = _append_case(cuda_device, 9, 2, 2, 128, 16, "head", 400, negative=0.0)
    n = kc.shape[0] * 16
    slots[2], slots[7] = n, 1 << 40
    kc0, vc0 = kc.clone(), vc.clone()
    fa.fa_paged_append(k, v, kc, vc, torch.as_tensor(slots, device=cuda_device))
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG and fa.fa_check_device_error() == fa.FA_OK
    slots[[2, 7]] = -1
    _check_append(kc0, vc0, kc, vc, slots, k, v, ref.f64(k), np.zeros(k.shape), 16, "append bad slot")


def test_side_streams(cuda_device):
    """Rotation and append on another stream than the current one, from tensors made there and here."""
    s = torch.cuda.Stream()
    q, k = _draw((2, 4, 200, 64), 450, cuda_device), _draw((2, 2, 200, 64), 451, cuda_device)
    freqs, pos = fa.fa_rope_freqs(64, device=cuda_device), torch.arange(200, dtype=torch.int32, device=cuda_device)
    want = fa.fa_rope(q, k, pos, freqs)
    kc, vc, slots, xq, xk, xv = _append_case(cuda_device, 200, 4, 2, 64, 16, "head", 452)
    st = torch.as_tensor(slots, device=cuda_device)
    kc2, vc2 = kc.clone(), vc.clone()
    wq = fa.fa_paged_append(xk, xv, kc, vc, st, q=xq, positions=pos, freqs=freqs)
    torch.cuda.synchronize()
    for _ in range(5):
        got = fa.fa_rope(q, k, pos, freqs, stream=s)
        back = fa.fa_rope_bwd(*got, pos, freqs, stream=s)
        gq = fa.fa_paged_append(xk, xv, kc2, vc2, st, q=xq, positions=pos, freqs=freqs, stream=s)
        del back
    s.synchronize()
    _ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(gq, wq) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_append_refusals(cuda_device):
    kc, vc, slots, q, k, v = _append_case(cuda_device, 9, 2, 2, 64, 16, "head", 500)
    st = torch.as_tensor(slots, device=cuda_device)
    freqs, pos = fa.fa_rope_freqs(64, device=cuda_device), torch.zeros(9, dtype=torch.int32, device=cuda_device)
    for bad in (dict(slots=st.int()), dict(slots=st[:8]), dict(k=k[:8]), dict(q=q[:8]), dict(v=v.float()),
                dict(v_cache=vc.float()), dict(v_cache=vc[:3]), dict(positions=pos), dict(freqs=freqs),
                dict(positions=pos[:8], freqs=freqs), dict(q_out=q), dict(k=torch.cat((k, k), 1)),
                dict(v_cache=vc.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(q=q, q_out=torch.empty(9, 4, 64, dtype=torch.bfloat16, device=cuda_device)[:, :2])):
        a = dict(k=k, v=v, k_cache=kc, v_cache=vc, slots=st)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            fa.fa_paged_append(**a)
    _ok()
