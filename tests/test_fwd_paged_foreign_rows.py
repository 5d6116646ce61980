"""A tile of query rows also holds rows that are not its unit's: the next sequence's queries, or places of q that no sequence has.
What lies there, NaN included, changes no bit of the unit's own results."""
import pytest
import torch

import attention_forward_05_gb300 as fa
from test_fwd_paged import Batch, many_places

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# d, chunks (context, new tokens): single tokens, drafts and short chunks whose rows leave most of a tile to others
SHAPES = [(64, [(1000, 1), (700, 3), (300, 1), (2000, 5)]), (128, [(1000, 1), (700, 3), (300, 1), (2000, 5)]),
          (128, [(1500, 23)]), (128, [(3000, 140), (900, 1)]), (64, [(3000, 140), (900, 1)])]


@pytest.mark.parametrize("window,sinks", [(0, 0), (400, 4)])
@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("d,chunks", SHAPES)
def test_places_behind_the_last_token(cuda_device, d, chunks, dealt, window, sinks):
    pad = many_places(8, 2) if dealt else 60
    b = Batch(cuda_device, 8, 2, d, 16, chunks, pad=pad, mult=3.0)
    b.q[b.T:] = 0
    want, want_l = b.run(window=window, sinks=sinks)
    b.check(want, want_l, f"d{d} dealt {dealt} window {window}", window=window, sinks=sinks)
    for junk in (float("nan"), float("inf"), -3e38, 1e4):
        b.q[b.T:] = junk
        o, lse = b.run(window=window, sinks=sinks)
        assert torch.equal(o[:b.T], want[:b.T]) and torch.equal(lse[:b.T], want_l[:b.T]), junk


@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("d,chunks", [s for s in SHAPES if len(s[1]) > 1])
def test_other_sequences(cuda_device, d, chunks, dealt):
    pad = many_places(8, 2) if dealt else 0
    b = Batch(cuda_device, 8, 2, d, 16, chunks, pad=pad, mult=3.0)
    b.q[b.T:] = 0
    want, want_l = b.run()
    first = 0
    for n in b.news:  # each sequence's queries as they are, all others spoiled
        for junk in (float("nan"), 1e4):
            q = torch.full_like(b.q, junk)
            q[first:first + n] = b.q[first:first + n]
            o, lse = b.run(q=q)
            assert torch.equal(o[first:first + n], want[first:first + n]), junk
            assert torch.equal(lse[first:first + n], want_l[first:first + n]), junk
        first += n
    assert fa.fa_check_device_error() == fa.FA_OK
