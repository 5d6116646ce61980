"""A serving loop's step with nothing to do: no new tokens and no sequences.  fa_rope, fa_paged_append and the decode calls
all take it, launch nothing and give empty results."""
import pytest
import torch

import attention_forward_05_gb300 as fa

pytestmark = pytest.mark.gpu


def _empty(*shape, dev, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=dev)


def _ok():
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("B,N", [(0, 5), (2, 0), (0, 0)])
def test_rotation_of_no_tokens(cuda_device, B, N, dtype):
    q, k = (_empty(B, h, N, 64, dev=cuda_device, dtype=dtype) for h in (4, 2))
    freqs = fa.fa_rope_freqs(64, device=cuda_device)
    for pos in (_empty(N, dev=cuda_device, dtype=torch.int32), _empty(B, N, dev=cuda_device, dtype=torch.int32),
                _empty(3, B, N, dev=cuda_device, dtype=torch.int32)):
        for call in (fa.fa_rope, fa.fa_rope_bwd):
            a, b = call(q, k, pos, freqs)
            assert a.shape == q.shape and b.shape == k.shape and a.dtype == b.dtype == dtype
            a, b = call(q, None, pos, freqs)
            assert a.shape == q.shape and b is None
            c, d = call(q, k, pos, freqs, None, False, q, k)
            assert c is q and d is k
    with pytest.raises((ValueError, fa.FAError)):  # still checked
        fa.fa_rope(q, k, _empty(N + 1, dev=cuda_device, dtype=torch.int32), freqs)
    _ok()


@pytest.mark.parametrize("prefix_len", [0, 20])
def test_step_without_sequences(cuda_device, prefix_len):
    kc = torch.randn(8, 2, 16, 64, device=cuda_device).to(torch.bfloat16)
    vc, before = kc.clone(), kc.clone()
    x = _empty(0, 4 + 2 * 2, 64, dev=cuda_device)
    freqs, pos = fa.fa_rope_freqs(64, device=cuda_device), _empty(0, dev=cuda_device, dtype=torch.int32)
    slots = _empty(0, dev=cuda_device, dtype=torch.int64)
    table, pre = _empty(0, 4, dev=cuda_device, dtype=torch.int32), torch.arange(2, dtype=torch.int32, device=cuda_device)
    for stream in (None, torch.cuda.Stream()):
        q = fa.fa_paged_append(x[:, 4:6], x[:, 6:], kc, vc, slots, q=x[:, :4], positions=pos, freqs=freqs, stream=stream)
        assert q.shape == (0, 4, 64)
        o, lse = fa.fa_decode_paged_prefix(q, kc, vc, pre, prefix_len, table, pos, with_lse=True, stream=stream)
        assert o.shape == (0, 4, 64) and lse.shape == (0, 4) and lse.dtype == torch.float32
        given = _empty(0, 4, 64, dev=cuda_device)
        o, none = fa.fa_decode_paged(q, kc, vc, table, pos, o=given, stream=stream)
        assert o is given and none is None
    for bad in (dict(seq_lens=torch.zeros(1, dtype=torch.int32, device=cuda_device)), dict(q=_empty(0, 3, 64, dev=cuda_device)),
                dict(page_table=_empty(1, 4, dev=cuda_device, dtype=torch.int32))):
        with pytest.raises(ValueError):
            fa.fa_decode_paged(**{**dict(q=q, k_cache=kc, v_cache=vc, page_table=table, seq_lens=pos), **bad})
    _ok()
    assert torch.equal(kc, before) and torch.equal(vc, before)
