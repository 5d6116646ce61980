"""Bookkeeping, normed append and paged attention together, as a program that serves runs them: prompts in pieces, then single
tokens, captured and replayed, against a float64 model of the whole history."""
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref
from paged_ref import f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("d,window", [(64, 0), (128, 0), (128, 40)])
def test_steps(cuda_device, d, window):
    B, H, Hkv, ps, width, sinks = 3, 4, 2, 16, 16, 3
    dev = cuda_device
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    kc = torch.full((40, Hkv, ps, d), float("nan"), dtype=BF, device=dev)
    vc = torch.full_like(kc, float("inf"))
    table = torch.full((B, width), -5, dtype=torch.int32, device=dev)
    free = torch.randperm(40, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(dev)
    count, lens = i32([40]), i32([0] * B)
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g, device=dev)).to(BF) for _ in range(2))
    freqs = fa.fa_rope_freqs(d)
    # pieces of prompts beside single tokens; one place unused now and then
    steps = [[50, 0, 7], [33, 20, 1], [1, 1, 1], [1, 0, 40], [1, 1, 1], [1, 1, 1]]
    T = 90
    qkv, new = torch.zeros(T, H + 2 * Hkv, d, dtype=BF, device=dev), i32([0] * B)

    def step():
        cu, pos, slots, _, _ = fa.fa_paged_slots(lens, new, table, free, count, ps, T, seq_lens=lens, free_left=count)
        q = fa.fa_paged_append(qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kc, vc, slots, q=qkv[:, :H], positions=pos, freqs=freqs,
                               q_weight=wq, k_weight=wk)
        o, lse = fa.fa_fwd_paged(q, kc, vc, table, cu, lens, window=window, sinks=sinks, with_lse=True)
        return q, o, lse

    ws_graph, out = None, None
    past = [([], [], []) for _ in range(B)]  # q, k, v of each sequence so far, in float64
    for number, counts in enumerate(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device=dev).to(BF))
        new.copy_(i32(counts))
        if number < 2:
            out = step()
        else:  # captured once, replayed from then on
            if ws_graph is None:
                state = [t.clone() for t in (kc, vc, table, count, lens)]
                ws_graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(ws_graph):
                    out = step()
                for t, s in zip((kc, vc, table, count, lens), state):
                    assert torch.equal(t.nan_to_num(), s.nan_to_num())  # capturing runs nothing
            ws_graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_OK
        q, o, lse = out
        first = 0
        for b, n in enumerate(counts):
            ctx = len(past[b][1])
            rows = f64(qkv[first:first + n])
            pos = np.arange(ctx, ctx + n)[None]
            for x, w, at in ((rows[:, :H], wq, 0), (rows[:, H:H + Hkv], wk, 1)):
                y, _ = ref.norm_rope(x, f64(w), 1e-6, pos, f64(freqs), np.zeros(d // 2, int))
                # what the kernels hold is rounded to bf16
                past[b][at].extend(torch.as_tensor(y).to(BF).double().numpy())
            past[b][2].extend(rows[:, H + Hkv:])
            seen = ref.visible(ctx, n, window, sinks)
            for h in range(H if n else 0):
                qh = np.array([r[h] for r in past[b][0][ctx:]])
                k, v = (np.array([r[h // 2] for r in past[b][i]]) for i in (1, 2))
                ro, rl, to, tl = ref.attend(qh, k, v, seen, 1 / math.sqrt(d))
                # q and k may have been rounded the other way where they lie between two values: a bf16 step of each
                ds = 2.0 ** -7 / math.sqrt(d) * (np.abs(qh) @ np.abs(k).T).max(-1, keepdims=True) * 0.25
                e = np.abs(f64(o[first:first + n, h]) - ro)
                assert (e <= to + 2 * ds * np.abs(v).max()).all(), (number, b, h, e.max())
                assert (np.abs(f64(lse[first:first + n, h]) - rl) <= tl + ds[:, 0]).all()
            first += n
    assert lens.tolist() == [sum(c[b] for c in steps) for b in range(B)]
    assert count.item() == 40 - sum(-(-n // ps) for n in lens.tolist())
