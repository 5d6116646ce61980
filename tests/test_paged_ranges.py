"""The paged decode over wide tables, which are taken by CTAs that share all tiles (ranges) and joined by a second kernel:
many sequences, batches without a key, captured steps and the C entry points' own workspaces.  And kernels that directly
follow one another, with nothing between them that would wait: append, decode and decode through one workspace.

Which form a call takes shows in fa_decode_paged_call_bytes: without a prefix, ranges need a workspace, clusters none."""
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import paged_ref as ref

pytestmark = pytest.mark.gpu

WIDE = 40_000  # keys that a wide table has room for


def _ok():
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK


def _ranges(B, H, Hkv, d, ps, width):
    return fa.fa_decode_paged_call_bytes(B, H, Hkv, d, ps, width) > 0


def _randn(shape, dev, seed, mult=1.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * mult).to(torch.bfloat16)


def _int32(x, dev):
    return torch.as_tensor(np.asarray(x, np.int32), device=dev)


def _case(dev, lens, H, Hkv, d, ps, seed, prefix_len=0, room=WIDE):
    tables, prefix, total = ref.deal_pages(lens, ps, seed, extra=-(-prefix_len // ps))
    kc, vc = ref.paged_cache(total, Hkv, ps, d, dev, seed + 1)
    width = max(max(map(len, tables)), -(-room // ps), 1)
    table = ref.page_table(tables, dev, width, 1 << 29)
    if room:
        assert _ranges(len(lens), H, Hkv, d, ps, width)
    return dict(q=_randn((len(lens), H, d), dev, seed + 2, 1.5), kc=kc, vc=vc, tables=tables, prefix=prefix, plen=prefix_len,
                table=table, lens=lens, lens_t=_int32(lens, dev), prefix_t=_int32(prefix, dev))


def _run(c, q=None, lens=None, **kw):
    q, lens = c["q"] if q is None else q, c["lens_t"] if lens is None else lens
    if c["plen"]:
        return fa.fa_decode_paged_prefix(q, c["kc"], c["vc"], c["prefix_t"], c["plen"], c["table"], lens, with_lse=True, **kw)
    return fa.fa_decode_paged(q, c["kc"], c["vc"], c["table"], lens, with_lse=True, **kw)


def _check(c, o, lse, name, **kw):
    ref.check_decode(c["q"], c["kc"], c["vc"], o, lse, c["tables"], c["lens"], 1 / math.sqrt(c["q"].shape[-1]), name,
                     c["prefix"], c["plen"], **kw)


@pytest.mark.parametrize("d,prefix_len", [(64, 0), (128, 0), (64, 100)])
@pytest.mark.parametrize("share", [0.5, 0.0], ids=["half empty", "all with keys"])
def test_more_sequences_than_ctas_and_threads(cuda_device, d, prefix_len, share):
    """Thousands of sequences: several a thread of the plan and several a CTA of the outputs of empty ones."""
    rng = np.random.default_rng(5000)
    lens = np.where(rng.random(3001) < share, rng.choice([0, -1], 3001), rng.choice([1, 1, 2, 17, 40], 3001))
    c = _case(cuda_device, lens.tolist(), 2, 1, d, 16, 5001, prefix_len)
    o, lse = _run(c)
    _ok()
    _check(c, o, lse, f"{len(lens)} sequences d{d}", seqs=sorted({0, 1, 2, 2999, 3000, *rng.integers(0, 3001, 150).tolist()}))
    none = torch.as_tensor(lens < 0 if prefix_len else lens <= 0, device=cuda_device)
    assert (o[none] == 0).all() and (lse[none] == -math.inf).all() and torch.isfinite(lse[~none]).all()


@pytest.mark.parametrize("prefix_len", [0, 77])
@pytest.mark.parametrize("lens", [[0], [-5], [0, -1, 0], [-1] * 700, [0] * 500 + [3]], ids=lambda x: f"{len(x)} of {x[-1]}")
def test_batches_without_a_key(cuda_device, lens, prefix_len):
    """No tile at all, or one sequence with keys at the end of many without."""
    c = _case(cuda_device, lens, 8, 2, 64, 16, 5100 + len(lens), prefix_len)
    want = torch.full_like(c["q"], math.nan)
    o, lse = _run(c, o=want)
    _ok()
    _check(c, o, lse, f"{len(lens)} without keys", seqs=sorted({0, len(lens) // 2, len(lens) - 1}))
    if not prefix_len and max(lens) <= 0:
        assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("prefix_len", [0, 333])
def test_captured_steps_follow_the_device_lengths(cuda_device, prefix_len):
    """A step (append, decode over wide tables) captured twice and replayed while lengths, slots and positions move on in
    device memory: the plan reads the lengths of each replay.  They cross tile borders and go from none to some."""
    B, H, Hkv, d, ps, steps = 5, 8, 2, 64, 16, 24
    start = [0, 5, 120, 250, 1900]
    c = _case(cuda_device, [n + steps for n in start], H, Hkv, d, ps, 5200, prefix_len)
    xs = _randn((steps, B, H + 2 * Hkv, d), cuda_device, 5201)
    freqs = fa.fa_rope_freqs(d, device=cuda_device)

    def state():
        return dict(kc=c["kc"].clone(), vc=c["vc"].clone(), x=torch.zeros_like(xs[0]), lens=_int32(start, cuda_device))

    def step(s):
        x, n = s["x"], s["lens"]
        slot = c["table"].gather(1, (n // ps).long()[:, None])[:, 0].long() * ps + n % ps
        q = fa.fa_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], s["kc"], s["vc"], slot, q=x[:, :H], positions=n + prefix_len,
                               freqs=freqs)
        n += 1
        return fa.fa_decode_paged_prefix(q, s["kc"], s["vc"], c["prefix_t"], prefix_len, c["table"], n, with_lse=True)

    e, eager = state(), []
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
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(s)
        s["kc"].copy_(c["kc"]), s["vc"].copy_(c["vc"]), s["lens"].copy_(_int32(start, cuda_device))
        graphs.append((g, s, out))
    for i in range(steps):
        for g, s, out in graphs:
            s["x"].copy_(xs[i])
            g.replay()
            assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1]), i
    _ok()


@pytest.mark.parametrize("plen", [0, 300])
def test_c_abi_allocates_its_workspace(cuda_device, plen):
    """workspace = NULL where the call needs one: the C entry points take it stream-ordered, on the default and another
    stream and while a stream is captured, and give the binding's results."""
    L = fa.lib()
    c = _case(cuda_device, [500, 0, 33, -1, 9000], 8, 2, 128, 16, 5300 + plen, plen)
    B, W = c["table"].shape
    assert fa.fa_decode_paged_call_bytes(B, 8, 2, 128, 16, W, plen) > 0
    want, want_l = _run(c)
    torch.cuda.synchronize()
    pages, Hkv, ps, d = c["kc"].shape

    def call(o, lse, stream):
        head = [c["q"].data_ptr(), c["kc"].data_ptr(), c["vc"].data_ptr(), o.data_ptr()]
        tail = [c["table"].data_ptr(), W, c["lens_t"].data_ptr(), B, 8, Hkv, d, pages, ps, W, None, 128 ** -0.5, None, 0,
                lse.data_ptr(), stream.cuda_stream]
        if plen:
            return L.fa_decode_paged_prefix(*head, c["prefix_t"].data_ptr(), plen, *tail)
        return L.fa_decode_paged(*head, *tail)

    o, lse = torch.empty_like(want), torch.empty_like(want_l)
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        o.fill_(math.nan), lse.fill_(math.nan)
        torch.cuda.synchronize()
        assert call(o, lse, stream) == fa.FA_OK
        _ok()
        assert torch.equal(o, want) and torch.equal(lse, want_l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert call(o, lse, torch.cuda.current_stream()) == fa.FA_OK
    for _ in range(2):
        o.fill_(math.nan), lse.fill_(math.nan)
        g.replay()
        assert torch.equal(o, want) and torch.equal(lse, want_l)
    _ok()


# ------------------------------------------------------------------------------------------ nothing in between

def _same_without_pauses(reset, run, out):
    """run's calls, launched one behind the other and as one graph, give the bits that they give with a synchronisation
    after every call."""
    reset()
    run(torch.cuda.synchronize)
    _ok()
    want = out.clone()
    assert torch.isfinite(want.float()).all()
    for _ in range(4):
        reset()
        torch.cuda.synchronize()
        run(lambda: None)
        assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(lambda: None)
    for _ in range(4):
        reset()
        g.replay()
        assert torch.equal(out, want)
    _ok()


SHAPES = [(4, 8, 2, 64, 16, 0), (1, 16, 4, 128, 64, 0), (40, 32, 8, 128, 16, 1000), (64, 16, 4, 64, 24, 300),
          (3, 16, 2, 128, 5, 700)]


@pytest.mark.parametrize("room", [0, WIDE], ids=["clusters", "ranges"])
@pytest.mark.parametrize("B,H,Hkv,d,ps,prefix_len", SHAPES, ids=str)
def test_decode_directly_behind_append(cuda_device, room, B, H, Hkv, d, ps, prefix_len):
    """Steps of append and decode whose inputs are all made in advance: the decode (or the gather or prefix kernel in front
    of it) is launched as the append's programmatic dependent, the next append as the decode's."""
    steps = 30
    rng = np.random.default_rng(5400)
    start = rng.integers(0, 200, B)
    c = _case(cuda_device, (start + steps).tolist(), H, Hkv, d, ps, 5401, prefix_len, room)
    xs = _randn((steps, B, H + 2 * Hkv, d), cuda_device, 5402)
    lens = [_int32(start + i + 1, cuda_device) for i in range(steps)]
    pos = [_int32(start + i + prefix_len, cuda_device) for i in range(steps)]
    slots = [torch.as_tensor([int(t[n // ps]) * ps + n % ps for t, n in zip(c["tables"], start + i)], device=cuda_device)
             for i in range(steps)]
    freqs = fa.fa_rope_freqs(d, device=cuda_device)
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(B, H, Hkv, d, ps, prefix_len), dtype=torch.uint8, device=cuda_device)

    kc, vc = c["kc"].clone(), c["vc"].clone()
    q, out = torch.empty_like(xs[:, :, :H]).contiguous(), torch.empty((steps, B, H, d), dtype=xs.dtype, device=cuda_device)

    def reset():
        kc.copy_(c["kc"]), vc.copy_(c["vc"]), q.fill_(math.nan), out.fill_(math.nan)

    def run(pause):
        for i in range(steps):
            x = xs[i]
            fa.fa_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc, slots[i], q=x[:, :H], positions=pos[i], freqs=freqs,
                               q_out=q[i])
            pause()
            fa.fa_decode_paged_prefix(q[i], kc, vc, c["prefix_t"], prefix_len, c["table"], lens[i], workspace=ws, o=out[i])
            pause()

    _same_without_pauses(reset, run, out)


@pytest.mark.parametrize("room", [0, WIDE], ids=["clusters", "ranges"])
@pytest.mark.parametrize("B,H,Hkv,d,ps,prefix_len", SHAPES, ids=str)
def test_decodes_back_to_back_through_one_workspace(cuda_device, room, B, H, Hkv, d, ps, prefix_len):
    """Decodes of other queries and lengths directly one behind the other, with and without the prefix in turn, all through
    one workspace that each finds full of the last one's states."""
    steps = 24
    rng = np.random.default_rng(5500)
    longest = rng.integers(100, 700, B)
    c = _case(cuda_device, longest.tolist(), H, Hkv, d, ps, 5501, prefix_len, room)
    qs = _randn((steps, B, H, d), cuda_device, 5502, 1.5)
    lens = [_int32(rng.integers(-1, longest + 1), cuda_device) for _ in range(steps)]
    bytes_ = max(fa.fa_decode_paged_workspace_bytes(B, H, Hkv, d, ps, p) for p in (0, prefix_len))
    ws = torch.empty(bytes_, dtype=torch.uint8, device=cuda_device)

    out = torch.empty((steps, B, H, d), dtype=qs.dtype, device=cuda_device)

    def run(pause):
        for i in range(steps):
            plen = prefix_len if i % 3 else 0
            fa.fa_decode_paged_prefix(qs[i], c["kc"], c["vc"], c["prefix_t"], plen, c["table"], lens[i], workspace=ws,
                                      o=out[i])
            pause()

    _same_without_pauses(lambda: out.fill_(math.nan), run, out)
