"""An infinite or NaN element of a head in fa_norm_rope, its backward pass and the normed append: the definition gives
r = (mean(x^2) + eps)^(-1/2) = 0, so the head's other elements are zeros, the infinite one is inf * 0 = NaN, and NaN reaches the
element that it is rotated with, if there is one, and no other."""
import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref
from paged_ref import f64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS, N, PS = 1e-5, 9, 16


def draw(shape, dtype, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(dtype)


def spoiled(H, d, dtype, dev, seed):
    """[1, N, H, d], each head of each token with one infinite element, at another place in every head."""
    x = draw((1, N, H, d), dtype, seed, dev)
    t, h = torch.meshgrid(torch.arange(N, device=dev), torch.arange(H, device=dev), indexing="ij")
    x[0, t, h, (t * 29 + h * 37) % d] = float("inf")
    x[0, ::2] = -x[0, ::2]
    return x


def partner(index, rot, interleaved):
    """The element that `index` is rotated with, or itself."""
    if index >= rot:
        return index
    if interleaved:
        return index ^ 1
    return index + rot // 2 if index < rot // 2 else index - rot // 2


def check_head_by_head(got, x, rot, interleaved):
    """got, x [N, H, d]: NaN at the infinite element and its partner, zeros elsewhere."""
    got, x = f64(got), f64(x)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            at = int(np.flatnonzero(np.isinf(x[t, h]))[0])
            nan = {at, partner(at, rot, interleaved)}
            assert set(np.flatnonzero(np.isnan(got[t, h]))) == nan, (t, h, at, np.flatnonzero(np.isnan(got[t, h])))
            assert (np.delete(got[t, h], sorted(nan)) == 0).all(), (t, h, at)


def rotation(rot, dev):
    if not rot:
        return dict(positions=None, freqs=None)
    return dict(positions=torch.arange(5, 5 + N, dtype=torch.int32, device=dev), freqs=fa.fa_rope_freqs(rot, device=dev))


@pytest.mark.parametrize("H,Hkv", [(8, 2), (1, 0)])  # up to three heads take the lanes in another way
@pytest.mark.parametrize("d,rot,interleaved", [(64, 0, False), (64, 32, False), (64, 32, True), (64, 64, False), (128, 0, False),
                                               (128, 48, True), (128, 96, False), (128, 128, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(cuda_device, H, Hkv, d, rot, interleaved, dtype):
    q, k = spoiled(H, d, dtype, cuda_device, 1), spoiled(Hkv, d, dtype, cuda_device, 2) if Hkv else None
    wq, wk = draw((d,), dtype, 3, cuda_device), draw((d,), dtype, 4, cuda_device) if Hkv else None
    qo, ko = fa.fa_norm_rope(q.transpose(1, 2), None if k is None else k.transpose(1, 2), wq, wk, interleaved=interleaved, eps=EPS,
                             **rotation(rot, cuda_device))
    check_head_by_head(qo.transpose(1, 2)[0], q[0], rot, interleaved)
    if Hkv:
        check_head_by_head(ko.transpose(1, 2)[0], k[0], rot, interleaved)


@pytest.mark.parametrize("d,rot,interleaved", [(64, 0, False), (64, 32, True), (128, 96, False), (128, 128, False)])
def test_append(cuda_device, d, rot, interleaved):
    H, Hkv = 6, 2
    q, k, v = (spoiled(h, d, BF, cuda_device, i)[0] for i, h in enumerate((H, Hkv, Hkv)))
    wq, wk = draw((d,), BF, 3, cuda_device), draw((d,), BF, 4, cuda_device)
    kc, vc = (torch.zeros(1, Hkv, PS, d, dtype=BF, device=cuda_device) for _ in range(2))
    qo = fa.fa_paged_append(k, v, kc, vc, torch.arange(N, device=cuda_device), q=q, interleaved=interleaved, q_weight=wq, k_weight=wk,
                            eps=EPS, **rotation(rot, cuda_device))
    check_head_by_head(qo, q, rot, interleaved)
    check_head_by_head(kc[0].transpose(0, 1)[:N], k, rot, interleaved)
    assert torch.equal(vc[0].transpose(0, 1)[:N], v) and not kc[0, :, N:].any()


@pytest.mark.parametrize("rot", [0, 32, 64])
def test_backward(cuda_device, rot):
    """dx of a spoiled head is NaN as a whole (the mean is); dw gets NaN where some head's infinite element is; other heads keep
    their gradients."""
    d, H = 64, 4
    x = draw((1, N, H, d), F32, 1, cuda_device)
    x[0, 3, 1, 40] = float("inf")
    dy, w = draw((1, N, H, d), F32, 2, cuda_device), draw((d,), F32, 3, cuda_device)
    how = rotation(rot, cuda_device)
    dx, _, dw, _ = fa.fa_norm_rope_bwd(dy.transpose(1, 2), None, x.transpose(1, 2), None, w, None, eps=EPS, **how)
    dx = dx.transpose(1, 2)
    assert torch.isnan(dx[0, 3, 1]).all() and set(torch.isnan(dw).nonzero().flatten().tolist()) == {40}
    clean = torch.ones(1, N, H, dtype=torch.bool, device=cuda_device)
    clean[0, 3, 1] = False
    turn = (f64(how["positions"]).astype(int).reshape(1, 1, N), f64(how["freqs"]), np.zeros(rot // 2, int)) if rot else ()
    with np.errstate(invalid="ignore"):
        want, _, tol, _ = ref.norm_rope_bwd(f64(dy), f64(x), f64(w), EPS, *turn)
    keep = clean.cpu().numpy()
    ref.check(dx[clean], want[keep], tol[keep], "dx beside an infinite head")
