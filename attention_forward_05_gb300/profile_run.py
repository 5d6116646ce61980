"""Runs one kernel family on a named synthetic workload a few times (for profilers such as ncu).

    python -m attention_forward_05_gb300.profile_run --workload mh_prefill --launches 2
    python -m attention_forward_05_gb300.profile_run --workload decode --B 4 --launches 2
    python -m attention_forward_05_gb300.profile_run --workload mh_prefill --bwd --launches 2
    python -m attention_forward_05_gb300.profile_run --workload decode --B 8 --hkv 4 --launches 2
    python -m attention_forward_05_gb300.profile_run --op decode_paged --launches 2 --time

The first launch is a warm-up; the process exits 0 after a device synchronise
and a device-error check.  --B / --H override the workload's batch and heads
(keeping the per-head shapes) so that a capture can stay small.  --hkv N runs the
decode workload as grouped-query decode (fa_decode_splitkv_gqa) with N key/value
heads shared by its query heads.

--op runs a position or paged-cache operator instead of a workload, on inputs larger than L2 where nothing else is said:
  rope                 q and k of 4 x 4096 tokens, 16 + 16 heads of 64, bf16, read out of a projection's layout
  append               8191 tokens, 32 query and 8 key/value heads of 128, into pages of 64 rows
  decode_paged         32 sequences of 8192 keys, 32 query heads on 4 key/value heads of 128, pages of 16 rows
  decode_paged_prefix  the same heads: 16384 shared keys in pages of 64 rows, 256 sequences of 64 own keys
  norm_rope            norms and rotation of q and k of 2 x 8192 tokens, 32 + 8 heads of 128, bf16
  norm_rope_bwd        its gradients, the norms' weights' too
  norm_rope_fp32, norm_rope_bwd_fp32   the same in fp32
  append_norm          `append` with norms of the heads, into pages of 16 rows
  slots                page tables, positions and slots of 64 prompts of 1000 tokens behind 500
  fwd_paged            a prompt of 8191 tokens, 32 query heads on 8 key/value heads of 128, pages of 64 rows
  fwd_paged_d64        8 chunks of 512 tokens behind 4096 keys, 32 query heads on 4 of 64, pages of 16 rows
  fwd_paged_window     48 single tokens behind 8192 keys, window of 4096 and 4 sinks, 32 heads on 8 of 128, pages of 16
  fwd_paged_question   23 tokens behind 1000 keys, 32 heads on 8 of 128, pages of 16: a cluster of CTAs a unit (inputs in L2)
  fwd_paged_singles    128 single tokens behind 300 keys, the same heads: a CTA a unit, in waves
"""
from __future__ import annotations

import argparse
import dataclasses
import sys

import torch

import attention_forward_05_gb300 as fa
from attention_forward_05_gb300 import accounting
from attention_forward_05_gb300.inputs import WORKLOADS, make_dout, make_qkv, merge_order, workload_inputs


OPS = ("rope", "append", "decode_paged", "decode_paged_prefix", "norm_rope", "norm_rope_bwd", "slots", "fwd_paged",
       "fwd_paged_d64", "fwd_paged_window", "norm_rope_fp32", "norm_rope_bwd_fp32", "append_norm", "fwd_paged_question",
       "fwd_paged_singles")


def operator(name: str, dev):
    """(a call of the operator, its bytes, its FLOPs) on seeded inputs."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(1900 + OPS.index(name))

    dtype = torch.float32 if name.endswith("_fp32") else torch.bfloat16

    def draw(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(dtype)

    if name == "rope":
        B, N, H, d = 4, 4096, 16, 64
        q, k = draw(B, N, H, d).transpose(1, 2), draw(B, N, H, d).transpose(1, 2)
        pos, freqs = torch.arange(N, dtype=torch.int32, device=dev), fa.fa_rope_freqs(d, device=dev)
        return (lambda: fa.fa_rope(q, k, pos, freqs)), 2 * 2 * q.numel() * 2, 6 * q.numel()
    if name in ("append", "append_norm"):
        T, H, Hkv, d, ps = 8191, 32, 8, 128, 64 if name == "append" else 16
        x = draw(T, H + 2 * Hkv, d)
        pages = -(-T // ps)
        kc, vc = draw(pages, Hkv, ps, d), draw(pages, Hkv, ps, d)
        at = torch.arange(T, device=dev)
        slots = torch.randperm(pages, generator=gen, device=dev)[at // ps] * ps + at % ps
        pos, freqs = at.to(torch.int32), fa.fa_rope_freqs(d, device=dev)
        norms = {} if name == "append" else {"q_weight": draw(d), "k_weight": draw(d)}
        return (lambda: fa.fa_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc, slots, q=x[:, :H], positions=pos,
                                           freqs=freqs, **norms)), 4 * x.numel(), (8 if norms else 3) * T * (H + Hkv) * d
    if name.startswith("norm_rope"):
        B, N, H, Hkv, d = 2, 8192, 32, 8, 128
        q, k = draw(B, N, H, d).transpose(1, 2), draw(B, N, Hkv, d).transpose(1, 2)
        wq, wk, pos, freqs = draw(d), draw(d), torch.arange(N, dtype=torch.int32, device=dev), fa.fa_rope_freqs(d, device=dev)
        n, e = q.numel() + k.numel(), q.element_size()
        if "bwd" not in name:
            return (lambda: fa.fa_norm_rope(q, k, wq, wk, pos, freqs)), 2 * e * n, 8 * n
        dq, dk = draw(B, H, N, d), draw(B, Hkv, N, d)
        return (lambda: fa.fa_norm_rope_bwd(dq, dk, q, k, wq, wk, pos, freqs)), 3 * e * n, 16 * n
    if name == "slots":
        B, n, ctx, ps = 64, 1000, 500, 16
        pages = -(-(ctx + n) // ps)
        table = torch.zeros(B, pages, dtype=torch.int32, device=dev)
        free = torch.randperm(B * pages, generator=gen, device=dev).to(torch.int32)
        ctxs, news, count = (torch.full((m,), v, dtype=torch.int32, device=dev)
                             for m, v in ((B, ctx), (B, n), (1, B * pages)))
        return (lambda: fa.fa_paged_slots(ctxs, news, table, free, count, ps, B * n)), 12 * B * n, 0
    if name.startswith("fwd_paged"):
        B, n, ctx, H, Hkv, d, ps, window, sinks = {"fwd_paged": (1, 8191, 0, 32, 8, 128, 64, 0, 0),
                                                   "fwd_paged_d64": (8, 512, 4096, 32, 4, 64, 16, 0, 0),
                                                   "fwd_paged_window": (48, 1, 8191, 32, 8, 128, 16, 4096, 4),
                                                   "fwd_paged_question": (1, 23, 1000, 32, 8, 128, 16, 0, 0),
                                                   "fwd_paged_singles": (128, 1, 300, 32, 8, 128, 16, 0, 0)}[name]
        width = -(-(ctx + n) // ps)
        kc, vc = draw(B * width, Hkv, ps, d), draw(B * width, Hkv, ps, d)
        table = torch.randperm(B * width, generator=gen, device=dev).to(torch.int32).view(B, width)
        lens = torch.full((B,), ctx + n, dtype=torch.int32, device=dev)
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=dev)
        q = draw(B * n, H, d)
        keys = B * (window + sinks if window else ctx + n)
        pairs = keys if window else B * (n * ctx + n * (n + 1) // 2)
        return (lambda: fa.fa_fwd_paged(q, kc, vc, table, cu, lens, window=window, sinks=sinks)), \
            4 * keys * Hkv * d + 4 * q.numel(), 4 * H * d * pairs
    H, Hkv, d = 32, 4, 128
    B, n, ps, prefix = (32, 8192, 16, 0) if name == "decode_paged" else (256, 64, 64, 16384)
    width, shared = n // ps, prefix // ps
    pages = B * width + shared
    kc, vc = draw(pages, Hkv, ps, d), draw(pages, Hkv, ps, d)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table, pre = order[shared:].view(B, width), order[:shared].contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device=dev)
    q = draw(B, H, d)
    keys = B * n + prefix
    return (lambda: fa.fa_decode_paged_prefix(q, kc, vc, pre, prefix, table, lens)), 4 * keys * Hkv * d, \
        4 * H * d * B * (n + prefix)


def run_operator(a) -> int:
    fn, nbytes, flops = operator(a.op, torch.device("cuda:0"))
    fn()
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.launches):
        fn()
    end.record()
    torch.cuda.synchronize()
    if a.time and a.launches:
        ms = start.elapsed_time(end) / a.launches
        print(f"time: {a.op} {ms * 1e3:.1f} us/call {nbytes / ms / 1e6:.0f} GB/s {flops / ms / 1e9:.1f} TFLOP/s")
    if fa.fa_check_device_error() != fa.FA_OK:
        print("device error", file=sys.stderr)
        return 1
    print(f"ok: {a.op} launches={a.launches}")
    return 0


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", choices=sorted(WORKLOADS))
    ap.add_argument("--op", choices=OPS)
    ap.add_argument("--launches", type=int, default=2)
    ap.add_argument("--B", type=int, default=0)
    ap.add_argument("--H", type=int, default=0)
    ap.add_argument("--time", action="store_true", help="time the launches with CUDA events and print the rate")
    ap.add_argument("--causal", action="store_true", help="causal mask (prefill workloads)")
    ap.add_argument("--bwd", action="store_true", help="time the backward (fa_bwd) after one forward (prefill)")
    ap.add_argument("--hkv", type=int, default=0, help="decode: grouped-query decode with this many key/value heads")
    a = ap.parse_args(argv)
    if (a.workload is None) == (a.op is None):
        ap.error("one of --workload and --op")
    if a.op:
        return run_operator(a)
    w = WORKLOADS[a.workload]
    if a.B:
        w = dataclasses.replace(w, B=a.B)
    if a.H:
        w = dataclasses.replace(w, H=a.H)
    dev = torch.device("cuda:0")
    q, k, v = workload_inputs(w, device=dev)
    if a.hkv:
        if not w.splits or w.H % a.hkv:
            ap.error("--hkv takes the decode workload and a divisor of its head count")
        _, k, v = make_qkv(w.B, a.hkv, 1, w.Nk, w.d, w.dtype, seed=w.seed + a.hkv, device=dev)
    order = torch.as_tensor(merge_order(w.splits, w.order_seed), device=dev) if w.splits else None
    o = torch.empty_like(q) if not w.splits else None
    lse = torch.empty((w.B, w.H, w.Nq), device=dev) if not w.splits else None

    if a.bwd:
        if w.splits:
            ap.error("--bwd takes a prefill workload")
        dout = make_dout(w.B, w.H, w.Nq, w.d, w.dtype, seed=w.seed + 700, device=dev)
        fa.fa_fwd(q, k, v, scale=w.scale, o=o, lse=lse, causal=a.causal)
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
        ws = torch.empty(fa.fa_bwd_workspace_bytes(w.B, w.H, w.Nq, w.d), dtype=torch.uint8, device=dev)

    def run():
        if a.bwd:
            fa.fa_bwd(q, k, v, o, dout, lse, scale=w.scale, causal=a.causal, dq=grads[0], dk=grads[1], dv=grads[2],
                      workspace=ws)
        elif a.hkv:
            fa.fa_decode_splitkv_gqa(q, k, v, w.splits, merge_order=order)
        elif w.splits:
            fa.fa_decode_splitkv_ex(q, k, v, w.splits, merge_order=order)
        else:
            fa.fa_fwd(q, k, v, scale=w.scale, o=o, lse=lse, causal=a.causal)

    torch.cuda.synchronize()
    run()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.launches):
        run()
    end.record()
    torch.cuda.synchronize()
    if a.time and a.launches:
        ms = start.elapsed_time(end) / a.launches
        if a.bwd:
            fl = accounting.bwd_flops_causal(w.B, w.H, w.Nq, w.Nk, w.d) if a.causal else \
                accounting.bwd_flops(w.B, w.H, w.Nq, w.Nk, w.d)
            rate = f"{fl / ms / 1e9:.1f} TFLOP/s (backward{', causal' if a.causal else ''})"
        elif a.hkv:
            rate = f"{accounting.decode_gqa_min_bytes(w.B, w.H, a.hkv, w.Nk, w.d) / ms / 1e6:.1f} GB/s"
        elif w.splits:
            rate = f"{accounting.decode_min_bytes(w.B, w.H, w.Nk, w.d) / ms / 1e6:.1f} GB/s"
        elif a.causal:
            rate = f"{accounting.fwd_flops_causal(w.B, w.H, w.Nq, w.Nk, w.d) / ms / 1e9:.1f} TFLOP/s (causal)"
        else:
            rate = f"{accounting.fwd_flops(w.B, w.H, w.Nq, w.Nk, w.d) / ms / 1e9:.1f} TFLOP/s"
        print(f"time: {w.name} {ms * 1e3:.1f} us/launch {rate}")
    if fa.fa_check_device_error() != fa.FA_OK:
        print("device timeout", file=sys.stderr)
        return 1
    hkv = f" Hkv={a.hkv}" if a.hkv else ""
    print(f"ok: {w.name} B={w.B} H={w.H}{hkv} Nq={w.Nq} Nk={w.Nk} d={w.d} launches={a.launches}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
