"""Bookkeeping, normed append and paged attention together, each part held to its own bound.

Nothing is allowed for what an earlier part rounded: queries and cached keys are compared with the float64 norms and rotations of
the whole history, cached values bit for bit, and then o and lse with the float64 attention of the very bf16 tensors that the kernel
read.  So a wrong slot, page, position or key shows (the last test plants such mistakes in the reference)."""
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref
from paged_ref import f64

BF = torch.bfloat16
EPS = 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d,ps,rot,inter,window,sinks", [
    (4, 2, 64, 16, 64, False, 0, 0), (8, 2, 128, 16, 128, False, 0, 0), (4, 2, 128, 24, 64, True, 40, 3), (6, 2, 64, 5, 32, False, 33, 0),
    (8, 1, 128, 64, 128, True, 100, 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_steps(cuda_device, H, Hkv, d, ps, rot, inter, window, sinks, captured):
    dev, B, width = cuda_device, 4, -(-320 // ps)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    pages = 3 * width
    kc, vc = torch.full((pages, Hkv, ps, d), float("nan"), dtype=BF, device=dev), torch.full((pages, Hkv, ps, d), float("inf"), dtype=BF, device=dev)
    table = torch.full((B, width), -7, dtype=torch.int32, device=dev)
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(dev)
    count, lens, new = i32([pages]), i32([0] * B), i32([0] * B)
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g, device=dev)).to(BF) for _ in range(2))
    freqs = fa.fa_rope_freqs(rot, device=dev)
    steps = [[50, 0, 7, 120], [33, 20, 1, 0], [1, 1, 1, 1], [0, 90, 40, 1], [1, 1, 1, 100], [ps, 1, 0, 1], [1, 1, 1, 1]]
    T = 190
    qkv = torch.zeros(T, H + 2 * Hkv, d, dtype=BF, device=dev)

    def step():
        cu, pos, slots, _, _ = fa.fa_paged_slots(lens, new, table, free, count, ps, T, seq_lens=lens, free_left=count)
        q = fa.fa_paged_append(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kc, vc, slots, q=qkv[:, :H], positions=pos, freqs=freqs,
                               interleaved=inter, q_weight=wq, k_weight=wk, eps=EPS)
        return q, cu, *fa.fa_fwd_paged(q, kc, vc, table, cu, lens, window=window, sinks=sinks, with_lse=True)

    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
    past = [np.zeros((0, H + 2 * Hkv, d)) for _ in range(B)]  # each sequence's rows of qkv
    fr = f64(freqs)
    for number, counts in enumerate(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=dev).to(BF))
        new.copy_(i32(counts))
        if graph is None:
            out = step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_OK
        q, cu, o, lse = out
        rows, tables = f64(qkv), table.tolist()
        first = np.concatenate([[0], np.cumsum(counts)]).tolist()
        assert cu.tolist() == first
        held = []
        for b, n in enumerate(counts):
            past[b] = np.concatenate([past[b], rows[first[b]:first[b] + n]])
            total = len(past[b])
            at = np.arange(total)
            how = (at[None], fr, np.zeros(rot // 2, int), inter)
            want_q, tol_q = ref.norm_rope(past[b][:, :H], f64(wq), EPS, *how)
            if n:
                ref.check(q[first[b]:first[b] + n], want_q[total - n:], tol_q[total - n:], f"step {number}: q of sequence {b}")
            if total:
                pg = np.asarray(tables[b], dtype=np.int64)[at // ps]
                assert (pg >= 0).all()
                held += sorted(set(pg.tolist()))
                row = torch.as_tensor(at % ps, device=dev)
                pg = torch.as_tensor(pg, device=dev)
                want_k, tol_k = ref.norm_rope(past[b][:, H:H + Hkv], f64(wk), EPS, *how)
                ref.check(kc[pg, :, row], want_k, tol_k, f"step {number}: keys of sequence {b}")
                assert np.array_equal(f64(vc[pg, :, row]), past[b][:, H + Hkv:]), f"step {number}: values of sequence {b}"
        assert len(held) == len(set(held)) == pages - count.item()  # no page twice, none lost
        assert lens.tolist() == [len(p) for p in past]
        ref.check_fwd_paged(q, kc, vc, tables, lens.tolist(), counts, o, lse, f"step {number}", window=window, sinks=sinks)


@pytest.mark.parametrize("keys", [10, 60, 300])
def test_the_bounds_notice_one_wrong_key(keys):
    """On data of the kind above: one key of a token's history left out, or exchanged for another key, is outside check_fwd_paged's
    bounds of o and of lse together, for nearly every key."""
    rng = np.random.default_rng(keys)
    d, noticed, tries = 64, 0, 0
    q, k, v = rng.normal(size=(8, d)), rng.normal(size=(keys, d)), rng.normal(size=(keys, d))
    seen = np.ones((8, keys), bool)
    o, lse, tol, tol_l = ref.attend(q, k, v, seen, 1 / math.sqrt(d))
    for j in range(0, keys, 3):
        hole = seen.copy()
        hole[:, j] = False
        k2, v2 = k.copy(), v.copy()
        k2[j], v2[j] = k[j - 1], v[j - 1]
        for o2, lse2 in (ref.attend(q, k, v, hole, 1 / math.sqrt(d))[:2], ref.attend(q, k2, v2, seen, 1 / math.sqrt(d))[:2]):
            tries += 1
            # by all of the token's heads: one of the eight rows is enough
            noticed += bool((np.abs(o2 - o) > tol).any() or (np.abs(lse2 - lse) > tol_l).any())
    assert noticed == tries
