"""Windows at least as long as any sequence, up to the largest int: the same bits as none, in both forms of the call."""
import pytest
import torch

from test_fwd_paged import MIXED, Batch, many_places

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("H,Hkv,d,ps", [(8, 2, 64, 16), (4, 1, 128, 32), (3, 1, 128, 1)])
def test_windows_of_any_length(cuda_device, H, Hkv, d, ps, dealt):
    b = Batch(cuda_device, H, Hkv, d, ps, MIXED, pad=many_places(H, Hkv) if dealt else 0)
    want, want_l = b.run()
    for window in (2 ** 20, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, 2 ** 31 - 1):
        for sinks in (0, 4, 2 ** 31 - 1):
            o, lse = b.run(window=window, sinks=sinks)
            assert torch.equal(o[:b.T], want[:b.T]) and torch.equal(lse[:b.T], want_l[:b.T]), (window, sinks)
    for window in (1, 100):  # first keys that are all keys
        o, lse = b.run(window=window, sinks=2 ** 31 - 1)
        b.check(o, lse, f"window {window}, all keys first", window=window, sinks=2 ** 31 - 1)
