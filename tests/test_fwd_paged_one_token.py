"""fa_fwd_paged on one token (or none): its token stride is never stepped over, so heads may lie as far apart as they like."""
import ctypes

import pytest
import torch

import attention_forward_05_gb300 as fa


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (4, 4)])
def test_strides_of_no_tokens_are_not_refused(H, Hkv):
    # T = 0 launches nothing, here or on a GPU: the call ends at its check of the device, behind those of the strides
    P = 0x10000
    for strides in ((0, 192), (8, 1 << 20), (H * 64, 64)):
        st = fa.lib().fa_fwd_paged(P, P, P, P, P, 4, P, P, 0, 2, H, Hkv, 64, 8, 16, 4, (ctypes.c_longlong * 2)(*strides), None, 0.125,
                                   0, 0, None, 0, None, None)
        assert st != fa.FA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 64), (2, 1, 64), (2, 2, 128), (6, 2, 128)])
def test_heads_far_apart(cuda_device, H, Hkv, d):
    from test_fwd_paged import Batch

    b = Batch(cuda_device, H, Hkv, d, 16, [(70, 1)])
    want, want_l = b.run()
    b.check(want, want_l, "one token")
    for apart in (d + 8, 3 * d, 50 * d):
        wide = torch.full((1, H, apart), float("nan"), dtype=torch.bfloat16, device=cuda_device)
        wide[..., :d] = b.q
        o, lse = b.run(q=wide[..., :d])
        assert torch.equal(o, want) and torch.equal(lse, want_l)
