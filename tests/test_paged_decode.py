"""GPU parity of fa_decode_paged and fa_decode_paged_prefix against the float64 definition (tests/paged_ref.py), and
of the position, cache and decode entry points run together."""
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import paged_ref as ref
from attention_forward_05_gb300.inputs import make_dout

pytestmark = pytest.mark.gpu


def _q(B, H, d, dev, seed, mult=1.5):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return (torch.randn((B, H, d), generator=g, device=dev) * mult).to(torch.bfloat16)


def _ok():
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK


# Keys that every table has room for.  Short tables are taken by one cluster of CTAs a unit, with no join after it;
# tables of 40000 keys by CTAs that share all tiles evenly.
MIN_TABLE = 0


@pytest.fixture(params=[0, 40_000], ids=["clusters", "ranges"])
def table_room(request, monkeypatch):
    monkeypatch.setitem(globals(), "MIN_TABLE", request.param)


def _case(dev, lens, H, Hkv, d, ps, seed, layout="head", prefix_len=0, spoil=True):
    tables, prefix, total = ref.deal_pages(lens, ps, seed, extra=-(-prefix_len // ps))
    kc, vc = ref.paged_cache(total, Hkv, ps, d, dev, seed + 1, layout)
    if spoil:
        ref.spoil_unused(kc, vc, tables, lens, prefix, prefix_len)
    return dict(q=_q(len(lens), H, d, dev, seed + 2), kc=kc, vc=vc, tables=tables, prefix=prefix, plen=prefix_len,
                table=ref.page_table(tables, dev, max(max(map(len, tables), default=1), -(-MIN_TABLE // ps), 1), 1 << 29),
                lens=lens,
                lens_t=torch.as_tensor(np.asarray(lens, np.int32), device=dev),
                prefix_t=torch.as_tensor(np.asarray(prefix, np.int32), device=dev))


def _run(c, scale=None, **kw):
    if c["plen"]:
        return fa.fa_decode_paged_prefix(c["q"], c["kc"], c["vc"], c["prefix_t"], c["plen"], c["table"], c["lens_t"],
                                         scale=scale, with_lse=True, **kw)
    return fa.fa_decode_paged(c["q"], c["kc"], c["vc"], c["table"], c["lens_t"], scale=scale, with_lse=True, **kw)


def _check(c, o, lse, name, scale=None, **kw):
    d = c["q"].shape[-1]
    ref.check_decode(c["q"], c["kc"], c["vc"], o, lse, c["tables"], c["lens"], scale or 1 / math.sqrt(d), name,
                     c["prefix"], c["plen"], **kw)


RAGGED = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 130, 300, -1, 511, 700]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (6, 2), (8, 1), (16, 2), (17, 1), (24, 2), (33, 1), (71, 1)], ids=str)
def test_groups(cuda_device, table_room, d, H, Hkv):
    c = _case(cuda_device, RAGGED, H, Hkv, d, 16, 1000 + H + d)
    o, lse = _run(c)
    _ok()
    _check(c, o, lse, f"paged d{d} H{H} Hkv{Hkv}")


@pytest.mark.parametrize("layout", ["head", "row", "one", "odd"])
@pytest.mark.parametrize("ps", [1, 5, 8, 16, 24, 64, 100, 256, 1024])
def test_pages_and_layouts(cuda_device, table_room, layout, ps):
    """Page sizes that divide a tile, span several or end inside one; contiguous and strided caches; unused rows and
    pages hold NaN and infinities, unused table entries numbers past the cache."""
    for d, lens in ((64, RAGGED), (128, [ps, ps + 1, max(1, ps - 1), 2 * ps, 333])):
        c = _case(cuda_device, lens, 8, 2, d, ps, 1100 + ps + d, layout)
        o, lse = _run(c)
        _ok()
        _check(c, o, lse, f"paged {layout} ps{ps} d{d}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [0], [-5], [40_000], [20_000, 3], [5, 9000, 0, 1, 4097]], ids=str)
def test_few_sequences(cuda_device, d, lens):
    """One or few sequences: the keys of one are split over the whole GPU."""
    c = _case(cuda_device, lens, 8, 2, d, 32, 1200 + d + len(lens), spoil=False)
    o, lse = _run(c)
    _ok()
    _check(c, o, lse, f"paged few d{d} {lens}", heads=[0, 5, 7])


@pytest.mark.parametrize("d,H,Hkv", [(128, 8, 1), (64, 16, 8)])
def test_many_sequences(cuda_device, d, H, Hkv):
    """A few hundred sequences of all lengths, empty ones among them; every head of sampled sequences."""
    rng = np.random.default_rng(1300)
    lens = np.exp(rng.uniform(0, math.log(3000), 301)).astype(int)
    lens[rng.random(301) < 0.1] = 0
    lens[rng.random(301) < 0.05] = -1
    c = _case(cuda_device, lens.tolist(), H, Hkv, d, 16, 1301, spoil=False)
    o, lse = _run(c)
    _ok()
    seqs = sorted({0, 1, 299, 300, *rng.integers(0, 301, 40).tolist()})
    _check(c, o, lse, f"paged many d{d}", seqs=seqs)
    empty = torch.as_tensor(lens <= 0, device=cuda_device)
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all() and torch.isfinite(lse[~empty]).all()


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.2, 1e-3])
def test_scales(cuda_device, table_room, scale):
    c = _case(cuda_device, [100, 1, 77], 4, 2, 64, 16, 1400)
    o, lse = _run(c, scale=scale)
    _ok()
    ref.check_decode(c["q"], c["kc"], c["vc"], o, lse, c["tables"], c["lens"], scale, f"scale {scale}")


@pytest.mark.parametrize("d,B", [(64, 3), (64, 40), (128, 3), (128, 40)])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_prefix_scales(cuda_device, table_room, scale, d, B):
    """Both tile widths of the prefix (B * 4 rows a head), its last tile ragged, infinities and NaN behind its end."""
    c = _case(cuda_device, [17 + b % 5 for b in range(B)], 8, 2, d, 16, 1430 + B, prefix_len=203)
    o, lse = _run(c, scale=scale)
    _ok()
    ref.check_decode(c["q"], c["kc"], c["vc"], o, lse, c["tables"], c["lens"], scale, f"prefix scale {scale} d{d} B{B}",
                     c["prefix"], 203)


@pytest.mark.parametrize("prefix_len", [0, 150])
def test_peaked_scores_and_late_maxima(cuda_device, table_room, prefix_len):
    """Scores that grow along the sequence by far more than a rescale threshold, and one key that outweighs all."""
    for d in (64, 128):
        c = _case(cuda_device, [900, 33, 257], 8, 2, d, 16, 1500 + d, prefix_len=prefix_len, spoil=False)
        for b, n in enumerate(c["lens"]):
            for i in range(n):
                c["kc"][int(c["tables"][b][i // 16]), :, i % 16] *= 1.0 + 9.0 * i / n
        c["kc"][int(c["tables"][1][2]), :, 0] = 40.0
        o, lse = _run(c)
        _ok()
        _check(c, o, lse, f"peaked d{d} prefix {prefix_len}")


def test_infinite_and_nan_keys_stay_in_their_sequence(cuda_device, table_room):
    """NaN or infinity in a key or value that a sequence does see makes that sequence's heads NaN (or infinite), as the
    formula does, and no other's."""
    c = _case(cuda_device, [70, 70, 70, 70], 4, 2, 64, 16, 1600)
    clean, _ = _run(c)
    c["kc"][int(c["tables"][1][2]), 0, 3] = math.nan
    c["vc"][int(c["tables"][2][1]), 1, 0] = math.inf
    o, lse = _run(c)
    _ok()
    assert torch.isnan(o[1, :2].float()).all() and torch.isnan(lse[1, :2]).all()
    assert not torch.isfinite(o[2, 2:].float()).any() and torch.isfinite(lse[2]).all()
    assert torch.equal(o[0], clean[0]) and torch.equal(o[3], clean[3])
    assert torch.equal(o[1, 2:], clean[1, 2:]) and torch.equal(o[2, :2], clean[2, :2])


@pytest.mark.parametrize("prefix_len", [0, 40])
def test_bad_pages_and_lengths(cuda_device, table_room, prefix_len):
    """A page outside the cache or a length past the table gives NaN in that sequence alone and is reported; nothing is
    read out of bounds (every index is checked before it is used)."""
    c = _case(cuda_device, [100, 64, 33, 16, 5], 8, 2, 128, 16, 1700, prefix_len=prefix_len)
    good, good_l = _run(c)
    _ok()
    c["table"][0, 3] = -1
    c["table"][2, 2] = c["kc"].shape[0]
    c["lens_t"][3] = c["table"].shape[1] * 16 + 1
    o, lse = _run(c)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG and fa.fa_check_device_error() == fa.FA_OK
    for b in (0, 2, 3):
        assert torch.isnan(o[b].float()).all() and torch.isnan(lse[b]).all(), b
    # the others: the work split may differ with the lengths, the values only by rounding
    c["lens"][3] = -1  # not looked at below
    _check(c, o, lse, "beside bad pages", seqs=[1, 4])


def test_bad_prefix_page(cuda_device, table_room):
    c = _case(cuda_device, [30, 0, -1, 50], 8, 2, 64, 16, 1750, prefix_len=200)
    c["prefix_t"][5] = 1 << 28
    o, lse = _run(c)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG and fa.fa_check_device_error() == fa.FA_OK
    assert torch.isnan(o[[0, 1, 3]].float()).all() and torch.isnan(lse[[0, 1, 3]]).all()
    assert (o[2] == 0).all() and (lse[2] == -math.inf).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,ps,prefix_len", [
    (1, 4, 4, 16, 1), (2, 8, 2, 16, 63), (3, 6, 2, 64, 64), (5, 16, 2, 16, 1000), (33, 8, 1, 32, 517), (40, 24, 2, 24, 300),
    (70, 4, 4, 5, 129), (64, 8, 2, 128, 2048), (9, 40, 1, 256, 100), (4, 8, 8, 8, 4000), (3, 4, 1, 1, 70),
    (150, 16, 4, 16, 700), (140, 4, 2, 5, 200), (90, 12, 4, 24, 333), (200, 16, 8, 8, 97)], ids=str)
def test_prefix(cuda_device, table_room, d, B, H, Hkv, ps, prefix_len):
    """Sequences with the prefix alone, with own rows behind it, and unused places; prefixes of one key, ending inside a
    page or a tile; batches below and above one tile of query rows."""
    rng = np.random.default_rng(1800 + B)
    lens = rng.integers(0, 150, B).tolist()
    if B > 3:
        lens[1], lens[2], lens[3] = 0, -1, 1
    c = _case(cuda_device, lens, H, Hkv, d, ps, 1801 + B + d, prefix_len=prefix_len)
    o, lse = _run(c)
    _ok()
    seqs = None if B < 12 else sorted({0, 1, 2, 3, B - 1, *rng.integers(0, B, 8).tolist()})
    _check(c, o, lse, f"prefix d{d} B{B} H{H}/{Hkv} ps{ps} P{prefix_len}", seqs=seqs)


@pytest.mark.parametrize("layout", ["row", "one", "odd"])
def test_prefix_layouts(cuda_device, table_room, layout):
    for d, ps in ((64, 16), (128, 64), (64, 100), (128, 12)):
        c = _case(cuda_device, [5, 80, 0], 8, 2, d, ps, 1900 + d, layout, prefix_len=333)
        o, lse = _run(c)
        _ok()
        _check(c, o, lse, f"prefix {layout} d{d} ps{ps}")


def test_prefix_equals_the_same_keys_in_every_table(cuda_device):
    """The shared-prefix decode and the paged decode whose tables name the prefix's pages agree within rounding, and with
    no sequence having own keys the result is the prefix's alone."""
    B, H, Hkv, d, ps, plen = 21, 16, 2, 128, 16, 512
    lens = np.random.default_rng(2000).integers(0, 90, B)
    c = _case(cuda_device, lens.tolist(), H, Hkv, d, ps, 2001, prefix_len=plen)
    o, lse = _run(c)
    whole = torch.cat((c["prefix_t"].expand(B, -1), c["table"]), 1).contiguous()
    o2, lse2 = fa.fa_decode_paged(c["q"], c["kc"], c["vc"], whole, c["lens_t"] + plen, with_lse=True)
    _ok()
    c["tables"] = [np.concatenate((c["prefix"], t)) for t in c["tables"]]
    c["lens"], c["plen"], c["prefix"] = (lens + plen).tolist(), 0, ()
    _check(c, o, lse, "prefix", seqs=[0, 7, 20])
    _check(c, o2, lse2, "whole tables", seqs=[0, 7, 20])
    # both are within the bound of one exact value, so within twice the bound of each other (P and O rounded to bf16)
    assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * o.float().abs().max().clamp(min=1.0)
    zero = torch.zeros_like(c["lens_t"])
    o3, _ = fa.fa_decode_paged_prefix(c["q"], c["kc"], c["vc"], c["prefix_t"], plen, c["table"], zero, with_lse=True)
    o4, _ = fa.fa_decode_paged(c["q"], c["kc"], c["vc"], whole, zero + plen, with_lse=True)
    _ok()
    assert (o3.float() - o4.float()).abs().max() <= 4 * 2.0 ** -8 * o3.float().abs().max().clamp(min=1.0)


def test_repeats_are_identical_and_caller_buffers(cuda_device, table_room):
    """Bit-identical repeats, into a caller's o with a caller's dirty workspace."""
    for plen in (0, 700):
        c = _case(cuda_device, [900, 20, 0, 4000, 1], 16, 2, 128, 16, 2100, prefix_len=plen)
        a, la = _run(c)
        need = fa.fa_decode_paged_workspace_bytes(5, 16, 2, 128, 16, plen)
        assert need > 0
        ws = torch.full((need,), 255, dtype=torch.uint8, device=cuda_device)
        o = torch.full((5, 16, 128), math.nan, dtype=torch.bfloat16, device=cuda_device)
        for _ in range(3):
            b, lb = _run(c, workspace=ws, o=o)
            assert b is o and torch.equal(a, b) and torch.equal(la, lb)
        _ok()


def test_workspace_that_is_too_small_is_refused(cuda_device, table_room):
    for plen, ps in ((0, 16), (700, 16), (90, 5)):
        c = _case(cuda_device, [90, 20], 16, 2, 128, ps, 2150, prefix_len=plen)
        need = fa.fa_decode_paged_workspace_bytes(2, 16, 2, 128, ps, plen)
        with pytest.raises(fa.FAError):
            _run(c, workspace=torch.empty(need - 256, dtype=torch.uint8, device=cuda_device))
        _run(c, workspace=torch.empty(need, dtype=torch.uint8, device=cuda_device))
        _ok()


@pytest.mark.parametrize("B,H,Hkv,d,ps,prefix_len", [
    (4, 8, 2, 64, 16, 0), (40, 32, 8, 128, 16, 1000), (64, 16, 4, 64, 24, 300), (3, 16, 2, 128, 5, 700)], ids=str)
def test_kernels_that_start_early_see_what_was_written(cuda_device, table_room, B, H, Hkv, d, ps, prefix_len):
    """Append, decode and two rotations in place, each on the one before's output, through one workspace: launched without
    a pause they give the bits that they give with a synchronisation after every call."""
    steps = 15
    tables, prefix, total = ref.deal_pages([200 + steps] * B, ps, 2900, extra=-(-prefix_len // ps))
    kc0, vc0 = ref.paged_cache(total, Hkv, ps, d, cuda_device, 2901)
    width = max(len(tables[0]), -(-MIN_TABLE // ps))
    table, pre = ref.page_table(tables, cuda_device, width, 1 << 28), torch.as_tensor(np.asarray(prefix, np.int32),
                                                                                    device=cuda_device)
    start = torch.as_tensor(np.random.default_rng(2902).integers(0, 200, B).astype(np.int32), device=cuda_device)
    freqs, x0 = fa.fa_rope_freqs(d, device=cuda_device), _q(B, H + 2 * Hkv, d, cuda_device, 2903)
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(B, H, Hkv, d, ps, prefix_len), dtype=torch.uint8, device=cuda_device)

    def run(pause):
        kc, vc, x, lens, out = kc0.clone(), vc0.clone(), x0, start.clone(), []
        for _ in range(steps):
            slot = table.gather(1, (lens // ps).long()[:, None])[:, 0].long() * ps + lens % ps
            q = fa.fa_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc, slot, q=x[:, :H], positions=lens + prefix_len,
                                   freqs=freqs)
            pause()
            lens += 1
            o, _ = fa.fa_decode_paged_prefix(q, kc, vc, pre, prefix_len, table, lens, workspace=ws)
            pause()
            o4, pos = o.view(B, H, 1, d), lens[:, None].contiguous()
            fa.fa_rope(o4, None, pos, freqs, q_out=o4)
            pause()
            fa.fa_rope_bwd(o4, None, pos, freqs, dq_in=o4)
            pause()
            x = torch.cat((o * 0.9 + x[:, :H] * 0.1, o[:, :2 * Hkv]), 1)
            out.append(x)
        _ok()
        return torch.stack(out)

    want = run(torch.cuda.synchronize)
    assert torch.isfinite(want.float()).all()
    for _ in range(3):
        assert torch.equal(run(lambda: None), want)


def test_short_tables_need_no_workspace(cuda_device):
    """fa_decode_paged_call_bytes: nothing for short tables, the whole workspace for long ones and behind a prefix; the C
    entry point takes a NULL workspace either way, also while a stream is being captured."""
    whole = fa.fa_decode_paged_workspace_bytes(3, 8, 2, 64, 16)
    assert whole > 0 and fa.fa_decode_paged_call_bytes(3, 8, 2, 64, 16, 0) == whole
    assert fa.fa_decode_paged_call_bytes(3, 8, 2, 64, 16, 8) == 0
    assert fa.fa_decode_paged_call_bytes(3, 8, 2, 64, 16, 4000) == whole
    behind = fa.fa_decode_paged_workspace_bytes(3, 8, 2, 64, 16, 100)
    assert fa.fa_decode_paged_call_bytes(3, 8, 2, 64, 16, 8, 100) == behind > whole
    c = _case(cuda_device, [90, 0, 33], 8, 2, 64, 16, 2170)
    want, want_l = _run(c)
    o, lse = torch.empty_like(want), torch.empty_like(want_l)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        st = fa.lib().fa_decode_paged(c["q"].data_ptr(), c["kc"].data_ptr(), c["vc"].data_ptr(), o.data_ptr(),
                                      c["table"].data_ptr(), c["table"].shape[1], c["lens_t"].data_ptr(), 3, 8, 2, 64,
                                      c["kc"].shape[0], 16, c["table"].shape[1], None, 0.125, None, 0, lse.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK
    for _ in range(2):
        o.fill_(math.nan)
        g.replay()
        assert torch.equal(o, want) and torch.equal(lse, want_l)
    _ok()


def test_side_stream_and_threads(cuda_device, table_room):
    """Calls on side streams, also from two host threads at once, give the results of the default stream."""
    import threading
    cases = [_case(cuda_device, [3000, 17, 0, 450], 8, 2, 64, 16, 2200 + i, prefix_len=500 * i) for i in range(2)]
    want = [_run(c) for c in cases]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            torch.cuda.set_device(cuda_device)
            s = torch.cuda.Stream()
            for _ in range(5):
                got[i].append(_run(cases[i], stream=s))
            s.synchronize()
        except Exception as e:
            errors.append(repr(e))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join(timeout=120)
        assert not t.is_alive()
    _ok()
    assert not errors
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("prefix_len", [0, 333])
def test_captured_steps_follow_the_device_lengths(cuda_device, prefix_len):
    """One generation step (append with rotation, then decode) captured into a graph and replayed while positions, slots
    and lengths move on in device memory: every replay equals the same step made eagerly.  Two graphs alternate."""
    B, H, Hkv, d, ps, steps = 4, 8, 2, 64, 16, 20
    start = [0, 5, 30, 14]
    tables, prefix, total = ref.deal_pages([n + steps for n in start], ps, 2300, extra=-(-prefix_len // ps))
    kc0, vc0 = ref.paged_cache(total, Hkv, ps, d, cuda_device, 2301)
    table, prefix_t = ref.page_table(tables, cuda_device), torch.as_tensor(np.asarray(prefix, np.int32), device=cuda_device)
    freqs = fa.fa_rope_freqs(d, device=cuda_device)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(2302)
    xs = torch.randn((steps, B, H + 2 * Hkv, d), generator=g, device=cuda_device).to(torch.bfloat16)

    def state():
        return dict(kc=kc0.clone(), vc=vc0.clone(), x=torch.zeros_like(xs[0]),
                    lens=torch.as_tensor(np.asarray(start, np.int32), device=cuda_device))

    def step(s):
        slot = table.gather(1, (s["lens"] // ps).long()[:, None])[:, 0].long() * ps + s["lens"] % ps
        x = s["x"]
        q = fa.fa_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], s["kc"], s["vc"], slot, q=x[:, :H],
                               positions=s["lens"] + prefix_len, freqs=freqs)
        s["lens"] += 1
        return fa.fa_decode_paged_prefix(q, s["kc"], s["vc"], prefix_t, prefix_len, table, s["lens"], with_lse=True)

    e = state()
    eager = []
    for i in range(steps):
        e["x"].copy_(xs[i])
        eager.append([t.clone() for t in step(e)])
    _ok()
    graphs = []
    for _ in range(2):
        s = state()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(s)
        torch.cuda.current_stream().wait_stream(side)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step(s)
        s["kc"].copy_(kc0), s["vc"].copy_(vc0), s["lens"].copy_(torch.as_tensor(start, device=cuda_device))
        graphs.append((gr, s, out))
    for i in range(steps):
        for gr, s, out in graphs:
            s["x"].copy_(xs[i])
            gr.replay()
            assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1]), i
    _ok()


def test_long_cache_offsets(cuda_device):
    """A cache of more than 2^31 elements, with sequences in its first and last pages."""
    Hkv, ps, d, H = 8, 64, 128, 16
    pages = (1 << 31) // (Hkv * ps * d) + 40
    kc = torch.zeros(pages, Hkv, ps, d, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.zeros_like(kc)
    small_k, small_v = ref.paged_cache(12, Hkv, ps, d, cuda_device, 2400)
    at = [pages - 1, 3, pages - 9, 0, pages - 20, pages - 2, 7, pages - 30, pages - 31, 11, pages - 3, pages - 4]
    kc[at], vc[at] = small_k, small_v
    tables = [np.asarray(at[:4]), np.asarray(at[4:7])]
    lens = [230, 130]
    prefix = np.asarray(at[7:])
    q = _q(2, H, d, cuda_device, 2401)
    table = ref.page_table(tables, cuda_device)
    lens_t = torch.as_tensor(np.asarray(lens, np.int32), device=cuda_device)
    for plen in (0, 300):
        o, lse = fa.fa_decode_paged_prefix(q, kc, vc, torch.as_tensor(prefix.astype(np.int32), device=cuda_device), plen,
                                           table, lens_t, with_lse=True)
        _ok()
        ref.check_decode(q, kc, vc, o, lse, tables, lens, 1 / math.sqrt(d), f"long cache P{plen}", prefix, plen)
    slots = torch.tensor([(pages - 5) * ps + 63, 5 * ps], device=cuda_device)
    k = _q(2, Hkv, d, cuda_device, 2402)
    fa.fa_paged_append(k, k * 2, kc, vc, slots)
    _ok()
    assert torch.equal(kc[pages - 5, :, 63], k[0]) and torch.equal(vc[5, :, 0], (k * 2)[1])
    assert int((kc[pages - 5] != 0).any(-1).sum()) == Hkv


def test_optional_results_and_views(cuda_device, table_room):
    """No LSE asked for; q with a token dimension; a table that is a slice of a wider one; prefix pages with
    more entries than the prefix needs; one sequence on one key/value head (strides of single entries)."""
    c = _case(cuda_device, [40, 0, 129], 8, 2, 64, 16, 2550, prefix_len=50)
    o, lse = _run(c)
    wide = torch.full((3, c["table"].shape[1] + 5), 1 << 29, dtype=torch.int32, device=cuda_device)
    wide[:, :c["table"].shape[1]] = c["table"]
    more = torch.cat((c["prefix_t"], torch.full((3,), -1, dtype=torch.int32, device=cuda_device)))
    o2, none = fa.fa_decode_paged_prefix(c["q"].unsqueeze(2), c["kc"], c["vc"], more, 50, wide[:, :c["table"].shape[1]],
                                         c["lens_t"])
    _ok()
    assert none is None and o2.shape == o.shape and torch.equal(o, o2)
    one = _case(cuda_device, [100], 4, 1, 128, 16, 2551)  # one sequence, one key/value head: strides of single entries
    a, _ = _run(one)
    t1 = one["table"].repeat(3, 1)[1:2]
    b, _ = fa.fa_decode_paged(one["q"], one["kc"], one["vc"], t1, one["lens_t"], with_lse=True)
    _ok()
    assert torch.equal(a, b)


def test_c_abi_allocates_its_workspace(cuda_device):
    """The C entry points with workspace = NULL and lse = NULL (stream-ordered allocation inside the call) give the
    binding's results, on the default and on another stream."""
    L = fa.lib()
    for plen in (0, 300):
        c = _case(cuda_device, [500, 0, 33, -1], 8, 2, 128, 16, 2560 + plen, prefix_len=plen)
        want, _ = _run(c)
        torch.cuda.synchronize()
        P, Hkv, ps, d = c["kc"].shape
        side = torch.cuda.Stream()
        for stream in (torch.cuda.current_stream(), side):
            o = torch.full((4, 8, 128), float("nan"), dtype=torch.bfloat16, device=cuda_device)
            torch.cuda.synchronize()
            args = [c["table"].data_ptr(), c["table"].shape[1], c["lens_t"].data_ptr(), 4, 8, Hkv, d, P, ps,
                    c["table"].shape[1], None, 128 ** -0.5, None, 0, None, stream.cuda_stream]
            if plen:
                st = L.fa_decode_paged_prefix(c["q"].data_ptr(), c["kc"].data_ptr(), c["vc"].data_ptr(), o.data_ptr(),
                                              c["prefix_t"].data_ptr(), plen, *args)
            else:
                st = L.fa_decode_paged(c["q"].data_ptr(), c["kc"].data_ptr(), c["vc"].data_ptr(), o.data_ptr(), *args)
            assert st == fa.FA_OK
            _ok()
            assert torch.equal(o, want)


def test_more_sequences_than_ctas_and_threads(cuda_device):
    """Thousands of sequences (several a thread of the plan), most of them empty or of one key."""
    rng = np.random.default_rng(2570)
    lens = rng.choice([0, 1, 1, 2, -1, 17, 40], 3001)
    c = _case(cuda_device, lens.tolist(), 2, 1, 64, 16, 2571, spoil=False)
    o, lse = _run(c)
    _ok()
    _check(c, o, lse, "3001 sequences", seqs=sorted({0, 1, 2, 3000, *rng.integers(0, 3001, 150).tolist()}))
    empty = torch.as_tensor(lens <= 0, device=cuda_device)
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all() and torch.isfinite(lse[~empty]).all()


def test_refusals(cuda_device):
    c = _case(cuda_device, [30, 4], 8, 2, 64, 16, 2500)
    base = dict(q=c["q"], k_cache=c["kc"], v_cache=c["vc"], page_table=c["table"], seq_lens=c["lens_t"])
    for bad in (dict(q=c["q"].float()), dict(q=c["q"][:, :7].contiguous()), dict(q=c["q"][:, ::2]), dict(q=c["q"][:1]),
                dict(k_cache=c["kc"].float()), dict(v_cache=c["vc"][:2]), dict(page_table=c["table"].long()),
                dict(page_table=c["table"][:1]), dict(page_table=c["table"][:, :0]), dict(seq_lens=c["lens_t"].long()),
                dict(seq_lens=c["lens_t"][:1]), dict(seq_lens=c["lens_t"].cpu()),
                dict(o=torch.empty(2, 8, 32, dtype=torch.bfloat16, device=cuda_device)),
                dict(page_table=c["table"].t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            fa.fa_decode_paged(**{**base, **bad})
    for bad in (dict(prefix_pages=None, prefix_len=4), dict(prefix_pages=c["table"][0], prefix_len=10_000),
                dict(prefix_pages=c["table"][0].long(), prefix_len=4), dict(prefix_pages=None, prefix_len=-1)):
        with pytest.raises((ValueError, TypeError)):
            fa.fa_decode_paged_prefix(**{**base, **bad})
    _ok()


def test_tensors_without_memory_are_refused(cuda_device):
    """Fake tensors pass every check of shape and device, and have no address: an exception, raised with the GIL held."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        q, cache = (torch.empty(s, dtype=torch.bfloat16, device=cuda_device) for s in ((2, 4, 64), (8, 2, 16, 64)))
        x, slots = torch.empty(2, 4, 3, 64, device=cuda_device), torch.empty(2, dtype=torch.int64, device=cuda_device)
        table, lens, pos = (torch.empty(s, dtype=torch.int32, device=cuda_device) for s in ((2, 4), (2,), (3,)))
        freqs = torch.empty(32, dtype=torch.float64, device=cuda_device)
    for call in (lambda: fa.fa_decode_paged(q, cache, cache, table, lens), lambda: fa.fa_rope(x, None, pos, freqs),
                 lambda: fa.fa_paged_append(q[:, :2], q[:, :2], cache, cache, slots)):
        with pytest.raises((RuntimeError, ValueError)):
            call()
    _ok()


# ------------------------------------------------------------------------------------------ together

def test_training_step_with_positions(cuda_device):
    """Rotation, causal attention, its backward and the rotation's backward, as a training step runs them (fp32): the
    gradients of the projections' outputs against central differences of the float64 loss."""
    B, H, Hkv, N, d = 1, 4, 2, 40, 64
    g = torch.Generator(device=cuda_device)
    g.manual_seed(2600)
    x = torch.randn((B, N, H + 2 * Hkv, d), generator=g, device=cuda_device)
    freqs = fa.fa_rope_freqs(d, device=cuda_device)
    pos = torch.arange(N, dtype=torch.int32, device=cuda_device) + 500
    q, k = fa.fa_rope(x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2), pos, freqs)
    v = x[:, :, H + Hkv:].transpose(1, 2).contiguous()
    o, lse = fa.fa_fwd(q, k, v, causal=True)
    dout = make_dout(B, H, N, d, "fp32", seed=2601, device=cuda_device)
    dq, dk, dv = fa.fa_bwd(q, k, v, o, dout, lse, causal=True)
    dq, dk = fa.fa_rope_bwd(dq, dk, pos, freqs)
    _ok()

    w, fr, axes = ref.f64(dout), ref.f64(freqs), np.zeros(d // 2, int)
    p = (np.arange(N) + 500)[None, None]
    x0 = ref.f64(x)

    def loss(y):
        yq, _ = ref.rotate(y[:, :, :H], p, fr, axes, False)
        yk, _ = ref.rotate(y[:, :, H:H + Hkv], p, fr, axes, False)
        total = 0.0
        for h in range(H):
            s = yq[0, :, h] @ yk[0, :, h // 2].T / 8.0
            s = np.where(np.tril(np.ones((N, N), bool)), s, -np.inf)
            e = np.exp(s - s.max(1, keepdims=True))
            total += ((e / e.sum(1, keepdims=True)) @ y[0, :, H + Hkv + h // 2] * w[0, h]).sum()
        return total

    rng = np.random.default_rng(2602)
    # the tf32 forward leaves errors of u = 2^-11 in O and LSE: 4u of each gradient's largest value bounds the backward
    # after it (tests/parity.py, the fp32 backward after the library's own forward); differences add h^2
    for grad, first, heads in ((dq, 0, H), (dk, H, Hkv), (dv, H + Hkv, Hkv)):
        top = grad.abs().max().item()
        for _ in range(12):
            h, n, e = rng.integers(heads), rng.integers(N), rng.integers(d)
            up, down = x0.copy(), x0.copy()
            up[0, n, first + h, e] += 1e-4
            down[0, n, first + h, e] -= 1e-4
            fd = (loss(up) - loss(down)) / 2e-4
            assert abs(fd - grad[0, h, n, e].item()) <= 4 * 2.0 ** -11 * top + 1e-6


def test_generation_matches_dense_attention(cuda_device):
    """A prompt's keys rotated and appended, then tokens generated one at a time for a ragged batch behind a shared
    prefix: each step's decode equals dense attention (fa_fwd) over the rows a sequence has, within rounding."""
    H, Hkv, d, ps, plen, steps = 8, 2, 128, 16, 75, 5
    lens = [0, 33, 200]
    B = len(lens)
    tables, prefix, total = ref.deal_pages([n + steps for n in lens], ps, 2700, extra=-(-plen // ps))
    kc, vc = ref.paged_cache(total, Hkv, ps, d, cuda_device, 2701)
    freqs = fa.fa_rope_freqs(d, device=cuda_device)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(2702)

    def draw(T):
        return torch.randn((T, H + 2 * Hkv, d), generator=g, device=cuda_device).to(torch.bfloat16)

    def slots_of(pages, first, n):
        return [int(pages[i // ps]) * ps + i % ps for i in range(first, first + n)]

    def append(x, slots, pos):
        return fa.fa_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc,
                                  torch.tensor(slots, dtype=torch.int64, device=cuda_device), q=x[:, :H],
                                  positions=torch.tensor(pos, dtype=torch.int32, device=cuda_device), freqs=freqs)

    shared = draw(plen)
    append(shared, slots_of(prefix, 0, plen), list(range(plen)))
    own = [draw(n) for n in lens]
    append(torch.cat(own), [s for b, n in enumerate(lens) for s in slots_of(tables[b], 0, n)],
           [plen + i for n in lens for i in range(n)])
    table, prefix_t = ref.page_table(tables, cuda_device), torch.as_tensor(np.asarray(prefix, np.int32), device=cuda_device)
    seen = [torch.cat((shared, x)) for x in own]
    for step in range(steps):
        x = draw(B)
        q = append(x, [slots_of(tables[b], lens[b] + step, 1)[0] for b in range(B)], [plen + n + step for n in lens])
        lens_t = torch.tensor([n + step + 1 for n in lens], dtype=torch.int32, device=cuda_device)
        o, lse = fa.fa_decode_paged_prefix(q, kc, vc, prefix_t, plen, table, lens_t, with_lse=True)
        _ok()
        for b in range(B):
            seen[b] = torch.cat((seen[b], x[b:b + 1]))
            n = seen[b].shape[0]
            y = seen[b][None]
            qd, kd = fa.fa_rope(y[:, :, :H].transpose(1, 2), y[:, :, H:H + Hkv].transpose(1, 2),
                                torch.arange(n, dtype=torch.int32, device=cuda_device), freqs)
            vd = y[:, :, H + Hkv:].transpose(1, 2).contiguous()
            od, ld = fa.fa_fwd(qd[:, :, -1:].contiguous(), kd, vd)
            _ok()
            assert torch.equal(qd[0, :, -1], q[b])  # the same rotation, bit for bit
            # both outputs are within one bf16 rounding of P and one of O of the same exact value
            assert (o[b].float() - od[0, :, 0].float()).abs().max() <= 4 * 2.0 ** -8 * vd.float().abs().max()
            assert (lse[b] - ld[0, :, 0]).abs().max() <= 1e-4
