"""fa_fwd_paged's workspace: small calls use none, dealt ones all of it; the C entry point's own one, and its default strides."""
import pytest
import torch

import attention_forward_05_gb300 as fa

BF = torch.bfloat16


def test_call_bytes_of_bad_arguments():
    good = (9, 2, 8, 2, 64, 16, 4)
    for at, bad in ((0, 0), (1, 0), (1, 16385), (2, 129), (3, 3), (4, 96), (5, 0), (6, 0), (6, 1 << 27)):
        assert fa.fa_fwd_paged_call_bytes(*good[:at], bad, *good[at + 1:]) == 0
    assert fa.fa_fwd_paged_call_bytes(*good, -1, 0) == 0 and fa.fa_fwd_paged_call_bytes(*good, 0, -1) == 0


SMALL = [(64, [(1000, 23)]), (128, [(1000, 23)]), (64, [(40, 3), (100, 1)]), (128, [(40, 3), (100, 1)])]
LARGE = [(64, [(5000, 200), (0, 900)]), (128, [(5000, 200), (0, 900)])]


def batch(dev, d, chunks):
    from test_fwd_paged import Batch

    return Batch(dev, 8, 2, d, 16, chunks, width=-(-max(c + n for c, n in chunks) // 16) * (1 if sum(n for _, n in chunks) < 30 else 200))


def sizes(b):
    return b.T, len(b.lens), *b.q.shape[1:2], b.kc.shape[1], b.q.shape[2]


@pytest.mark.gpu
@pytest.mark.parametrize("d,chunks", SMALL)
def test_small_calls_use_none(cuda_device, d, chunks):
    b = batch(cuda_device, d, chunks)
    assert fa.fa_fwd_paged_call_bytes(*sizes(b), 16, b.table.shape[1]) == 0 < fa.fa_fwd_paged_workspace_bytes(*sizes(b))
    b.run()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    o, lse = b.run()
    assert torch.cuda.max_memory_allocated() - before <= 2 * (o.nbytes + lse.nbytes) + 4096  # its results, and no more
    b.check(o, lse, "no workspace")
    for room in (16, 1 << 20):
        got = b.run(workspace=torch.empty(room, dtype=torch.uint8, device=cuda_device))
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)


@pytest.mark.gpu
@pytest.mark.parametrize("d,chunks", LARGE)
def test_dealt_calls_use_all(cuda_device, d, chunks):
    b = batch(cuda_device, d, chunks)
    need = fa.fa_fwd_paged_workspace_bytes(*sizes(b))
    assert fa.fa_fwd_paged_call_bytes(*sizes(b), 16, b.table.shape[1]) == need > 0
    want = b.run()
    got = b.run(workspace=torch.empty(need, dtype=torch.uint8, device=cuda_device))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(fa.FAError):
        b.run(workspace=torch.empty(need - 16, dtype=torch.uint8, device=cuda_device))


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 2)])
@pytest.mark.parametrize("d,chunks", SMALL + LARGE)
def test_c_entry_point_allocates_its_own(cuda_device, d, chunks, window, sinks):
    """workspace, strides and lse NULL: on the current stream, another one and under capture, as the binding's results."""
    b = batch(cuda_device, d, chunks)
    want, want_l = b.run(window=window, sinks=sinks)
    torch.cuda.synchronize()
    o, lse = torch.empty_like(want), torch.empty_like(want_l)

    def call(stream, with_lse):
        p = [t.data_ptr() for t in (b.q, b.kc, b.vc, o, b.table)]
        return fa.lib().fa_fwd_paged(*p, b.table.stride(0), b.cu.data_ptr(), b.len_t.data_ptr(), *sizes(b), b.kc.shape[0], 16,
                                     b.table.shape[1], None, None, d ** -0.5, window, sinks, None, 0,
                                     lse.data_ptr() if with_lse else None, stream.cuda_stream)

    def check(with_lse):
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_OK
        assert torch.equal(o, want) and (torch.equal(lse, want_l) if with_lse else torch.isnan(lse).all())

    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        for with_lse in (False, True):
            o.fill_(float("nan"))
            lse.fill_(float("nan"))
            torch.cuda.synchronize()
            assert call(stream, with_lse) == fa.FA_OK
            check(with_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        assert call(torch.cuda.current_stream(), True) == fa.FA_OK
    for _ in range(2):
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        g.replay()
        check(True)
