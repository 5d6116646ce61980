"""Rotation and append of inputs whose bytes exceed the L2 cache, which are cut differently from small ones: a token's bits
are those that it has in a small call."""
import pytest
import torch

import attention_forward_05_gb300 as fa

pytestmark = pytest.mark.gpu


def _randn(shape, dev, dtype, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(dtype)


@pytest.mark.parametrize("mb", [155, 210, 290])
@pytest.mark.parametrize("H,Hkv,d,dtype,inter", [
    (1, 0, 64, torch.bfloat16, False), (3, 0, 128, torch.bfloat16, True), (5, 0, 64, torch.float32, False),
    (16, 4, 128, torch.bfloat16, True), (16, 16, 64, torch.bfloat16, False), (9, 3, 128, torch.float32, False)], ids=str)
def test_rotation(cuda_device, mb, H, Hkv, d, dtype, inter):
    N = mb * 1_000_000 // (2 * (H + Hkv) * d * (2 if dtype == torch.bfloat16 else 4)) + 3
    x = _randn((1, N, H + Hkv, d), cuda_device, dtype, 7000 + H)
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:].transpose(1, 2) if Hkv else None
    pos = torch.randint(-1000, 1_000_000, (3, 1, N), device=cuda_device, dtype=torch.int32)
    freqs, axes = fa.fa_rope_freqs(d, device=cuda_device), torch.arange(d // 2, device=cuda_device, dtype=torch.int32) % 3
    qo, ko = fa.fa_rope(q, k, pos, freqs, axes=axes, interleaved=inter)
    step = -(-N // 16)
    for a in range(0, N, step):
        s = slice(a, a + step)
        qs, ks = fa.fa_rope(q[:, :, s], None if k is None else k[:, :, s], pos[:, :, s].contiguous(), freqs, axes=axes,
                            interleaved=inter)
        assert torch.equal(qo[:, :, s], qs) and (k is None or torch.equal(ko[:, :, s], ks)), a
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK


@pytest.mark.parametrize("mb", [155, 290])
@pytest.mark.parametrize("H,Hkv,d", [(32, 8, 128), (3, 1, 64), (0, 1, 128)], ids=str)
def test_append(cuda_device, mb, H, Hkv, d):
    ps, heads = 64, H + 2 * Hkv
    T = mb * 1_000_000 // (4 * heads * d) + 5
    x = _randn((T, heads, d), cuda_device, torch.bfloat16, 7100 + H)
    q, k, v = x[:, :H] if H else None, x[:, H:H + Hkv], x[:, H + Hkv:]
    pages = -(-T // ps)
    slots = torch.randperm(pages * ps, device=cuda_device)[:T]
    pos, freqs = torch.arange(T, device=cuda_device, dtype=torch.int32), fa.fa_rope_freqs(d, device=cuda_device)
    caches = [torch.zeros(pages, Hkv, ps, d, dtype=torch.bfloat16, device=cuda_device) for _ in range(4)]
    qo = fa.fa_paged_append(k, v, *caches[:2], slots, q=q, positions=pos, freqs=freqs)
    step = -(-T // 16)
    for a in range(0, T, step):
        s = slice(a, a + step)
        qs = fa.fa_paged_append(k[s], v[s], *caches[2:], slots[s], q=None if q is None else q[s], positions=pos[s],
                                freqs=freqs)
        assert q is None or torch.equal(qo[s], qs), a
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
