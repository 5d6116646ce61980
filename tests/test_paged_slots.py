"""fa_paged_slots against its rules, one sequence at a time."""
import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref

pytestmark = pytest.mark.gpu

JUNK = -77


def make(B, ps, width, ctx_hi, new_hi, seed, spare=5, short=0, pad=7):
    """(ctx, new, table, free, count, T): rows of the table hold a permutation's pages, junk behind them."""
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, B)
    new = rng.integers(-1, new_hi + 1, B)
    held = -(-ctx // ps)
    need = -(-(ctx + np.maximum(new, 0)) // ps) - held
    order = rng.permutation(held.sum() + need.sum() + spare + 1)
    table = np.full((B, width), JUNK, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = order[at:].astype(np.int32)
    count = len(free) - short
    return ctx.astype(np.int32), new.astype(np.int32), table, free, count, int(np.maximum(new, 0).sum()) + pad


def call(dev, ctx, new, table, free, count, ps, T, **kw):
    t = {n: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=dev) for n, x in
         (("ctx", ctx), ("new", new), ("table", table), ("free", free), ("count", [count]))}
    out = fa.fa_paged_slots(t["ctx"], t["new"], t["table"], t["free"], t["count"], ps, T, **kw)
    torch.cuda.synchronize()
    return t, out, fa.fa_check_device_error()


def compare(t, out, err, want):
    cu, pos, slots, lens, left, table, failed = want
    for name, got, exp in zip(("cu", "positions", "slots", "seq_lens", "free_left"), out, (cu, pos, slots, lens, [left])):
        assert got.tolist() == list(exp), name
    assert t["table"].tolist() == [list(r) for r in table]
    assert err == (fa.FA_ERR_INVALID_ARG if failed else fa.FA_OK)


@pytest.mark.parametrize("B,ps,ctx_hi,new_hi", [
    (1, 16, 0, 1), (1, 1, 5, 3), (3, 16, 100, 40), (37, 24, 500, 1), (256, 64, 4000, 1), (1000, 16, 50, 9), (2049, 16, 40, 3),
    (16384, 8, 3, 2), (5, 16, 20, 9000), (61, 1, 30, 60), (64, 128, 0, 700),
    (61, 16, 700, 4000), (700, 8, 90, 60), (3, 7, 11, 9001), (300, 24, 5, 100),
])
def test_equals_the_rules(cuda_device, B, ps, ctx_hi, new_hi):
    ctx, new, table, free, count, T = make(B, ps, -(-(ctx_hi + new_hi) // ps) + 1, ctx_hi, new_hi, B + ps)
    want = ref.slots(ctx, new, table, free, count, ps, T)
    assert not want[-1]
    compare(*call(cuda_device, ctx, new, table, free, count, ps, T), want)


@pytest.mark.parametrize("kind", ["pages", "table", "places", "negative", "count", "none"])
def test_sequences_that_do_not_fit(cuda_device, kind):
    ps, B = 16, 40
    ctx, new, table, free, count, T = make(B, ps, 30, 200, 150, 11)
    if kind == "pages":
        count = len(free) // 2
    elif kind == "table":
        table = np.ascontiguousarray(table[:, :14])  # sequences past 224 tokens
        ctx = np.minimum(ctx, 14 * ps)
    elif kind == "places":
        T = T // 2
    elif kind == "negative":
        ctx[[3, 17]] = -1
        new[3] = 5
    elif kind == "count":
        count = len(free) + 1
    else:
        count = 0
    want = ref.slots(ctx, new, table, free, count, ps, T)
    assert want[-1] and (kind in ("count", "none") or any(l >= c + n > c for l, c, n in zip(want[3], ctx, new)))
    compare(*call(cuda_device, ctx, new, table, free, count, ps, T), want)


def test_no_sequences_and_no_tokens(cuda_device):
    e = np.zeros((0,), dtype=np.int32)
    t, out, err = call(cuda_device, e, e, np.zeros((0, 4), np.int32), [3, 4, 5], 2, 16, 6)
    assert [x.tolist() for x in out] == [[0], [0] * 6, [-1] * 6, [], [2]] and err == fa.FA_OK
    t, out, err = call(cuda_device, [5, 9], [0, -3], [[1], [2]], e, 0, 16, 0)
    assert [x.tolist() for x in out] == [[0, 0, 0], [], [], [5, 9], [0]] and err == fa.FA_OK


def test_in_place_and_captured(cuda_device):
    """A captured step that counts on by itself: lengths and the free pages' count are written where they were read."""
    ps, B, steps = 4, 9, 23
    ctx, _, table, free, count, _ = make(B, ps, 40, 60, 0, 5, spare=B * 10)
    new = np.ones(B, np.int32)
    new[4] = 0
    t = {n: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=cuda_device)
         for n, x in (("ctx", ctx), ("new", new), ("table", table), ("free", free), ("count", [count]))}

    def step():
        return fa.fa_paged_slots(t["ctx"], t["new"], t["table"], t["free"], t["count"], ps, B, seq_lens=t["ctx"],
                                 free_left=t["count"])

    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        cu, pos, slots, lens, left = step()
    assert lens is t["ctx"] and left is t["count"]
    for _ in range(steps):
        want = ref.slots(ctx, new, table, free, count, ps, B)
        g.replay()
        torch.cuda.synchronize()
        compare(t, (cu, pos, slots, lens, left), fa.fa_check_device_error(), want)
        ctx, count, table = np.asarray(want[3], np.int32), want[4], np.asarray(want[5], np.int32)


def test_wide_rows_and_another_stream(cuda_device):
    ctx, new, table, free, count, T = make(50, 16, 12, 90, 60, 3)
    want = ref.slots(ctx, new, table, free, count, 16, T)
    wide = torch.full((50, 31), 5, dtype=torch.int32, device=cuda_device)
    wide[:, :12] = torch.as_tensor(table, device=cuda_device)
    i = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=cuda_device)  # noqa: E731
    args = (i(ctx), i(new), wide[:, :12], i(free), i([count]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = fa.fa_paged_slots(*args, 16, T, stream=s)
    s.synchronize()
    compare({"table": wide[:, :12]}, out, fa.fa_check_device_error(), want)
    assert (wide[:, 12:] == 5).all()


@pytest.mark.parametrize("aligned", [True, False])
def test_many_tokens_in_place(cuda_device, aligned):
    """A cluster of many CTAs that counts on in place, outputs on 16-byte boundaries or not, eager and captured."""
    ps, B = 16, 2500
    ctx, new, table, free, count, T = make(B, ps, 40, 300, 30, 17, pad=5)
    assert T > 20000
    want = ref.slots(ctx, new, table, free, count, ps, T)
    i = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=cuda_device)  # noqa: E731
    first = {"ctx": i(ctx), "table": i(table), "count": i([count])}
    fixed = i(new), i(free)
    room = torch.empty(T + 4, dtype=torch.int32, device=cuda_device), torch.empty(T + 4, dtype=torch.int64, device=cuda_device)
    at = 0 if aligned else 1
    out = dict(positions=room[0][at:at + T], slots=room[1][at:at + T])
    state = {n: t.clone() for n, t in first.items()}

    def step():
        return fa.fa_paged_slots(state["ctx"], fixed[0], state["table"], fixed[1], state["count"], ps, T, seq_lens=state["ctx"],
                                 free_left=state["count"], **out)

    got = step()
    torch.cuda.synchronize()
    compare(state, got, fa.fa_check_device_error(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(20):
        for n, t in first.items():
            state[n].copy_(t)
        for t in out.values():
            t.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        compare(state, got, fa.fa_check_device_error(), want)
