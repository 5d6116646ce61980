"""fa_fwd_paged against the float64 definition: ragged chunks, pages of any size, windows, sinks, odd heads."""
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import step_ref as ref
from paged_ref import deal_pages, page_table, paged_cache, spoil_unused

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Batch:
    """Chunks (context, new tokens) over a shuffled cache whose unused rows hold NaN and infinities."""

    def __init__(self, dev, H, Hkv, d, ps, chunks, layout="head", seed=1, pad=0, mult=1.5, width=None):
        self.news = [n for _, n in chunks]
        self.lens = [c + n for c, n in chunks]
        self.tables, _, pages = deal_pages(self.lens, ps, seed)
        self.kc, self.vc = paged_cache(pages, Hkv, ps, d, dev, seed, layout)
        spoil_unused(self.kc, self.vc, self.tables, self.lens)
        g = torch.Generator(device=dev)
        g.manual_seed(seed + 1)
        self.T = sum(self.news)
        self.q = (torch.randn((self.T + pad, H, d), generator=g, device=dev) * mult).to(BF)
        self.table = page_table(self.tables, dev, width)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.news)]), dtype=torch.int32, device=dev)
        self.len_t = torch.tensor(self.lens, dtype=torch.int32, device=dev)

    def run(self, q=None, **kw):
        return fa.fa_fwd_paged(self.q if q is None else q, self.kc, self.vc, self.table, self.cu, self.len_t,
                               **{"with_lse": True, **kw})

    def check(self, o, lse, name, **kw):
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_OK
        kw.pop("with_lse", None)
        ref.check_fwd_paged(self.q, self.kc, self.vc, self.tables, self.lens, self.news, o, lse, name, **kw)


MIXED = [(0, 1), (130, 1), (5, 7), (0, 300), (257, 0), (63, 65), (1000, 23), (127, 1), (0, 128), (128, 129)]


@pytest.mark.parametrize("H,Hkv,d,ps,chunks", [
    (1, 1, 64, 16, [(0, 1)]), (4, 1, 128, 16, [(0, 1)]), (8, 2, 64, 16, [(63, 1)]), (8, 2, 128, 64, [(128, 1)]),
    (4, 4, 64, 16, [(0, 64)]), (4, 4, 128, 16, [(0, 128)]), (2, 2, 128, 32, [(0, 257)]), (2, 2, 64, 128, [(0, 513)]),
    (8, 2, 64, 16, MIXED), (8, 2, 128, 16, MIXED), (6, 2, 64, 32, MIXED), (6, 2, 128, 24, MIXED), (5, 1, 128, 64, MIXED),
    (4, 4, 128, 128, MIXED), (3, 3, 64, 24, MIXED), (16, 1, 64, 8, MIXED), (7, 1, 64, 256, MIXED),
    (8, 2, 64, 1, MIXED), (8, 2, 128, 1, MIXED), (4, 2, 128, 20, MIXED), (4, 2, 64, 3, MIXED), (2, 1, 64, 100, MIXED),
    (32, 1, 128, 16, [(300, 9), (0, 17)]), (128, 1, 64, 16, [(77, 3), (0, 2)]), (100, 1, 128, 16, [(40, 5)]),
    (8, 8, 128, 16, [(3000, 5)]), (4, 2, 64, 16, [(5000, 3), (0, 1), (4000, 60)]),
    (64, 1, 128, 16, [(10, 900), (300, 800)]), (128, 2, 64, 32, [(0, 500), (40, 300), (7, 1)]), (2, 1, 64, 128, [(9000, 71), (6000, 1)]),
])
def test_chunks(cuda_device, H, Hkv, d, ps, chunks):
    b = Batch(cuda_device, H, Hkv, d, ps, chunks)
    b.check(*b.run(), f"H{H}/{Hkv} d{d} ps{ps}")


def many_places(H, Hkv):
    """Places of q behind the last token with which a call may have more units than are given CTAs of their own."""
    return 2600 * (128 // (H // Hkv)) // Hkv + 1


CHUNKS_BY_RANGES = [
    (1, 1, 64, 16, [(0, 1)]), (4, 1, 128, 16, [(0, 1)]), (8, 2, 64, 16, [(63, 1)]), (8, 2, 128, 64, [(128, 1)]),
    (4, 4, 64, 16, [(0, 64)]), (2, 2, 128, 32, [(0, 257)]), (8, 2, 64, 16, MIXED), (8, 2, 128, 16, MIXED),
    (6, 2, 128, 24, MIXED), (5, 1, 64, 64, MIXED), (3, 3, 64, 24, MIXED), (8, 2, 64, 1, MIXED), (4, 2, 128, 20, MIXED),
    (128, 1, 64, 16, [(77, 3), (0, 2)]), (100, 1, 128, 16, [(40, 5)])]


@pytest.mark.parametrize("H,Hkv,d,ps,chunks", CHUNKS_BY_RANGES)
def test_chunks_by_ranges(cuda_device, H, Hkv, d, ps, chunks):
    b = Batch(cuda_device, H, Hkv, d, ps, chunks, pad=many_places(H, Hkv))
    b.check(*b.run(), f"H{H}/{Hkv} d{d} ps{ps} dealt")


@pytest.mark.parametrize("d", [64, 128])
def test_one_sequence_by_clusters_of_each_size(cuda_device, d):
    # tables of 1, 2, ... key tiles: as many CTAs a unit, up to 16, and more than that
    for keys in (1, 64, 65, 129, 257, 385, 600, 1000, 1300, 2000, 2600, 4100):
        for H, Hkv in ((4, 1), (16, 8)):
            b = Batch(cuda_device, H, Hkv, d, 16, [(keys - 1, 1)] if keys < 9 else [(keys - 9, 9)])
            b.check(*b.run(), f"{keys} keys, {Hkv} heads")


@pytest.mark.parametrize("B", [31, 32, 33, 90])
def test_more_sequences_by_clusters(cuda_device, B):
    # a warp, or the block, finds the unit; some sequences have no new tokens
    for d in (64, 128):
        b = Batch(cuda_device, 4, 1, d, 16, [((37 * i) % 300, (0, 1, 3, 2)[i % 4]) for i in range(B)])
        b.check(*b.run(), f"{B} sequences d{d}")


def test_both_forms_agree(cuda_device):
    # the same call with more places for tokens: another form, the same result but for the order of its sums
    for d in (64, 128):
        a = Batch(cuda_device, 8, 2, d, 16, [(900, 5), (0, 3), (130, 40)])
        o, lse = a.run()
        q = torch.zeros(a.T + many_places(8, 2), 8, d, dtype=BF, device=cuda_device)
        q[:a.T] = a.q
        o2, lse2 = a.run(q=q)
        torch.cuda.synchronize()
        # two results of the formula, each within check_fwd_paged's bound of it: P and o rounded to bf16, 2^-8 each
        assert (o.float() - o2[:a.T].float()).abs().max() <= 2 * 2 ** -7 * a.vc.float().nan_to_num(0, 0, 0).abs().max()
        assert (lse - lse2[:a.T]).abs().max() < 1e-4  # sums of 940 fp32 numbers in two orders: 940 * 2^-24, and ex2's 2^-22


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (128, 4), (129, 130), (500, 64), (100000, 0), (200, 100000)])
@pytest.mark.parametrize("H,Hkv,d,ps", [(8, 2, 64, 16), (4, 1, 128, 32), (3, 1, 128, 1), (2, 2, 64, 24)])
def test_windows(cuda_device, H, Hkv, d, ps, window, sinks):
    b = Batch(cuda_device, H, Hkv, d, ps, MIXED + [(2000, 1), (1500, 200)], seed=window)
    b.check(*b.run(window=window, sinks=sinks), f"window {window} sinks {sinks}", window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(1, 1), (7, 3), (64, 0), (129, 130), (500, 64)])
@pytest.mark.parametrize("H,Hkv,d,ps", [(8, 2, 64, 16), (4, 1, 128, 32), (3, 1, 128, 1)])
def test_windows_by_ranges(cuda_device, H, Hkv, d, ps, window, sinks):
    b = Batch(cuda_device, H, Hkv, d, ps, MIXED, pad=many_places(H, Hkv))
    b.check(*b.run(window=window, sinks=sinks), f"w{window} s{sinks} dealt", window=window, sinks=sinks)


def test_pages_behind_the_window_may_be_gone(cuda_device):
    """Pages that no token sees: junk in the table, NaN and infinities in their rows' neighbours."""
    for d, ps, window, sinks in ((64, 16, 100, 5), (128, 16, 300, 0), (128, 64, 70, 64), (64, 1, 33, 2)):
        b = Batch(cuda_device, 4, 2, d, ps, [(900, 40), (1300, 1), (20, 3)], seed=d + ps)
        keep = [ref.visible(n - m, m, window, sinks).any(0) for n, m in zip(b.lens, b.news)]
        for i, seen in enumerate(keep):
            for j, s in enumerate(seen):
                if not s:
                    b.kc[int(b.tables[i][j // ps]), :, j % ps] = float("nan")
                    b.vc[int(b.tables[i][j // ps]), :, j % ps] = float("inf")
            for p in range(len(b.tables[i])):
                if not seen[p * ps:(p + 1) * ps].any():
                    b.table[i, p] = -123456 if p % 2 else 2 ** 31 - 1
        b.check(*b.run(window=window, sinks=sinks), f"freed pages d{d} ps{ps}", window=window, sinks=sinks)


@pytest.mark.parametrize("layout", ["row", "one", "odd"])
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 64), (128, 20)])
def test_cache_layouts(cuda_device, layout, d, ps):
    b = Batch(cuda_device, 8, 2, d, ps, MIXED, layout=layout, seed=4)
    b.check(*b.run(), f"{layout} d{d} ps{ps}")


@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 64), (6, 2, 128), (1, 1, 128)])
def test_strided_queries(cuda_device, H, Hkv, d):
    b = Batch(cuda_device, H, Hkv, d, 16, MIXED)
    wide = torch.full((b.T, H + 3, d), float("nan"), dtype=BF, device=cuda_device)
    wide[:, 2:2 + H] = b.q
    b.check(*b.run(q=wide[:, 2:2 + H]), "slice of a projection")
    odd = torch.full((b.T, H, d + 8), float("nan"), dtype=BF, device=cuda_device)
    odd[..., :d] = b.q
    b.check(*b.run(q=odd[..., :d]), "padded heads")


def test_rows_behind_the_last_sequence_stay(cuda_device):
    for d in (64, 128):
        b = Batch(cuda_device, 4, 2, d, 16, [(10, 3), (200, 130)], pad=29)
        o = torch.full((b.T + 29, 4, d), 7.0, dtype=BF, device=cuda_device)
        lse = torch.full((b.T + 29, 4), 7.0, device=cuda_device)
        got = b.run(o=o, lse=lse)
        assert got[0] is o and got[1] is lse
        b.check(o, lse, "padded")
        assert (o[b.T:] == 7).all() and (lse[b.T:] == 7).all()


@pytest.mark.parametrize("scale", [0.0, -0.5, 1.0, 30.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(cuda_device, scale, d):
    b = Batch(cuda_device, 4, 2, d, 16, [(300, 40), (0, 200)], mult=0.7)
    b.check(*b.run(scale=scale), f"scale {scale}", scale=scale)


def test_growing_maxima(cuda_device):
    """Scores that grow with the key's place, so that every tile moves the maximum."""
    for d in (64, 128):
        b = Batch(cuda_device, 4, 2, d, 16, [(700, 150)])
        at = torch.arange(b.lens[0], device=cuda_device)
        pg = torch.as_tensor(np.asarray(b.tables[0], dtype=np.int64), device=cuda_device)[at // 16]
        b.kc[pg, :, at % 16, 0] = (at.float() * 0.25).to(BF)[:, None]
        b.q[..., 0] = 8.0
        b.check(*b.run(), "growing")


def test_values_of_later_tokens_do_not_reach_earlier_ones(cuda_device):
    """Infinite and NaN values of a key are seen by the tokens that see the key, and by no other."""
    for d, ps in ((64, 16), (128, 16), (128, 1)):
        for window in (0, 50):
            b = Batch(cuda_device, 4, 2, d, ps, [(100, 90), (30, 4)], seed=9)
            want, _ = b.run(window=window)
            key = 100 + 37
            b.vc[int(b.tables[0][key // ps]), :, key % ps, 5] = float("inf")
            b.vc[int(b.tables[0][key // ps]), :, key % ps, 9] = float("nan")
            o, _ = b.run(window=window)
            seen = torch.as_tensor(ref.visible(100, 90, window, 0)[:, key], device=cuda_device)
            assert seen.any() and not seen.all()
            assert (o[:90][seen][..., 5] == float("inf")).all() and torch.isnan(o[:90][seen][..., 9]).all()
            keep = torch.ones(94, 4, d, dtype=torch.bool, device=cuda_device)
            keep[:90][seen] = False
            assert torch.isfinite(o[keep]).all()
            assert (o[keep].float() - want[keep].float()).abs().max() <= 2 ** -7 * want[keep].float().abs().max()


def test_infinite_values_and_bad_sequences_by_ranges(cuda_device):
    for d, ps in ((64, 16), (128, 16), (128, 1)):
        b = Batch(cuda_device, 4, 2, d, ps, [(100, 90), (30, 4), (20, 7)], seed=9, pad=many_places(4, 2))
        want, _ = b.run()
        for key in (100 + 37, 100 + 70):
            b.vc[int(b.tables[0][key // ps]), :, key % ps, 5] = float("inf")
        b.len_t[2] = 3  # fewer keys than new tokens
        o, lse = b.run()
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG
        assert (o[37:90, :, 5] == float("inf")).all() and torch.isnan(o[94:101]).all() and torch.isnan(lse[94:101]).all()
        keep = torch.ones(94, 4, d, dtype=torch.bool, device=cuda_device)
        keep[37:90, :, 5] = False
        assert torch.isfinite(o[:94][keep]).all()
        assert (o[:94][keep].float() - want[:94][keep].float()).abs().max() <= 2 ** -7 * want[:94][keep].float().abs().max()


def test_bad_sequences_get_nan_and_others_nothing(cuda_device):
    for d in (64, 128):
        chunks = [(40, 6), (0, 5), (300, 20), (17, 1), (64, 3)]
        b = Batch(cuda_device, 4, 2, d, 16, chunks, width=25)
        b.len_t[1] = 3  # fewer keys than new tokens
        b.len_t[3] = 25 * 16 + 1  # more than the table holds
        b.table[2, 1] = b.kc.shape[0]
        o, lse = b.run()
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG
        first = np.concatenate([[0], np.cumsum(b.news)])
        for i in range(5):
            rows = slice(first[i], first[i + 1])
            if i in (1, 2, 3):
                assert torch.isnan(o[rows]).all() and torch.isnan(lse[rows]).all(), i
        b.check(o, lse, "beside bad ones", seqs={0, 4})  # the split of the work, and so the last bit, depends on all lengths


@pytest.mark.parametrize("cu,good", [([0, 6, 40, 31], [0]), ([0, 6, 11, 32], [0, 1]), ([-1, 6, 11, 31], [1, 2]),
                                     ([0, 2 ** 30, 11, 31], [2]), ([0, 6, 11, 2 ** 31 - 1], [0, 1]), ([7, 6, 11, 31], [1, 2])])
def test_bad_offsets_write_nothing_of_their_sequence(cuda_device, cu, good):
    for d in (64, 128):
        b = Batch(cuda_device, 4, 2, d, 16, [(40, 6), (0, 5), (30, 20)])
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        o = torch.full((31, 4, d), 7.0, dtype=BF, device=cuda_device)
        b.run(o=o)
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG
        for i, rows in enumerate((slice(0, 6), slice(6, 11), slice(11, 31))):
            if i not in good:
                assert (o[rows] == 7).all(), i
        b.check(o, None, "beside bad ones", seqs=set(good))


def test_offsets_of_far_too_many_blocks_write_nothing(cuda_device):
    # 0, T, 0, T, ...: every other sequence has all tokens, more blocks than T tokens can have in as many sequences
    T, B = 600, 4000
    for d in (64, 128):
        q = torch.zeros(T, 2, d, dtype=BF, device=cuda_device)
        cache = torch.zeros(4, 1, 16, d, dtype=BF, device=cuda_device)
        cu = torch.arange(B + 1, dtype=torch.int32, device=cuda_device) % 2 * T
        table = torch.zeros(B, 50, dtype=torch.int32, device=cuda_device)
        lens = torch.full((B,), 700, dtype=torch.int32, device=cuda_device)
        o = torch.full((T, 2, d), 7.0, dtype=BF, device=cuda_device)
        fa.fa_fwd_paged(q, cache, cache, table, cu, lens, o=o)
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == fa.FA_ERR_INVALID_ARG
        assert (o == 7).all()


def test_no_tokens_and_no_sequences(cuda_device):
    b = Batch(cuda_device, 4, 2, 64, 16, [(40, 0), (0, 0)])
    o, lse = b.run()
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    q = torch.zeros(5, 4, 64, dtype=BF, device=cuda_device)
    o = torch.full((5, 4, 64), 7.0, dtype=BF, device=cuda_device)
    b.run(q=q, o=o)
    e = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    fa.fa_fwd_paged(q, b.kc, b.vc, e.view(0, 1), torch.zeros(1, dtype=torch.int32, device=cuda_device), e, o=o)
    torch.cuda.synchronize()
    assert (o == 7).all() and fa.fa_check_device_error() == fa.FA_OK


def test_same_bits_on_streams_graphs_and_workspaces(cuda_device):
    for d, chunks in ((64, MIXED), (128, MIXED), (128, [(4000, 9)])):
        b = Batch(cuda_device, 8, 2, d, 16, chunks)
        want = b.run()
        torch.cuda.synchronize()
        n = fa.fa_fwd_paged_workspace_bytes(b.T, len(b.lens), 8, 2, d)
        spaces = [torch.full((max(n, 16),), 255, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
        s = torch.cuda.Stream()
        other = b.run(stream=s)
        s.synchronize()
        outs = [other, b.run(workspace=spaces[0]), b.run(workspace=spaces[0])]
        for ws in spaces:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = b.run(workspace=ws)
            for t in out:
                t.zero_()
            g.replay()
            g.replay()
            outs.append(out)
            torch.cuda.synchronize()
        for got in outs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        b.check(*want, "shared")


def test_lengths_change_under_a_captured_graph(cuda_device):
    b = Batch(cuda_device, 8, 2, 128, 16, [(500, 30), (20, 30), (100, 30)])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = b.run(window=0)
    for lens, cu in (([530, 50, 130], [0, 30, 60, 90]), ([400, 1, 33], [0, 70, 71, 90]), ([530, 50, 130], [0, 0, 1, 90])):
        b.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        g.replay()
        b.lens, b.news = lens, [y - x for x, y in zip(cu, cu[1:])]
        b.check(o, lse, "replayed")


def test_single_tokens_equal_the_decode(cuda_device):
    """The chunk form of a decode batch against fa_decode_paged: the same definition, two kernels."""
    for d in (64, 128):
        b = Batch(cuda_device, 16, 4, d, 16, [(n, 1) for n in (0, 1, 15, 16, 500, 2047, 3000)])
        o, lse = b.run()
        od, ld = fa.fa_decode_paged(b.q, b.kc, b.vc, b.table, b.len_t, with_lse=True)
        b.check(o, lse, "single")
        assert (lse - ld).abs().max() <= 1e-5
        assert (o.float() - od.float()).abs().max() <= 2 ** -6 * od.float().abs().max()


def test_many_short_sequences(cuda_device):
    rng = np.random.default_rng(3)
    for d, B in ((64, 700), (128, 300), (128, 1500)):
        chunks = [(int(c), int(n)) for c, n in zip(rng.integers(0, 60, B), rng.integers(0, 4, B))]
        b = Batch(cuda_device, 4, 2, d, 16, chunks)
        b.check(*b.run(), f"{B} sequences", seqs=set(rng.integers(0, B, 60).tolist()) | {0, B - 1})


def test_the_most_sequences(cuda_device):
    """16384 places of a padded batch, nearly all unused; the used ones among them, the first and the last."""
    for d, window in ((64, 0), (128, 20)):
        chunks = [(0, 0)] * 16384
        used = {0: (5, 3), 1: (0, 1), 700: (100, 40), 8191: (17, 1), 16382: (0, 300), 16383: (33, 2)}
        for i, c in used.items():
            chunks[i] = c
        b = Batch(cuda_device, 4, 2, d, 16, chunks, width=20)
        b.len_t[[i for i in range(16384) if i not in used]] = -1
        b.check(*b.run(window=window, sinks=2), "16384 places", seqs=set(used), window=window, sinks=2)


def test_a_long_prompt(cuda_device):
    for H, Hkv, d, n in ((4, 2, 128, 3001), (2, 2, 64, 2500)):
        b = Batch(cuda_device, H, Hkv, d, 64, [(0, n)])
        b.check(*b.run(), f"prompt of {n}")
        dense = [x[torch.as_tensor(np.asarray(b.tables[0], dtype=np.int64), device=cuda_device)].transpose(0, 1).flatten(1, 2)[:, :n]
                 for x in (b.kc, b.vc)]
        o, _ = fa.fa_fwd(b.q.transpose(0, 1)[None].contiguous(), dense[0][None].contiguous(), dense[1][None].contiguous(),
                         causal=True)
        got, _ = b.run()
        assert (o[0].transpose(0, 1).float() - got.float()).abs().max() <= 2 ** -6 * o.float().abs().max()


def test_a_long_cache_past_32_bit_offsets(cuda_device):
    """Pages whose elements lie past 2^31 of the cache's start."""
    pages, ps, d = 2 ** 31 // (128 * 128) + 70, 128, 128  # over 2^31 elements a cache
    kc = torch.zeros(pages, 1, ps, d, dtype=BF, device=cuda_device)
    vc = torch.zeros_like(kc)
    ids = [pages - 1, 3, pages - 7, pages - 50]
    g = torch.Generator(device=cuda_device)
    g.manual_seed(3)
    for i in ids:
        kc[i] = torch.randn((1, ps, d), generator=g, device=cuda_device).to(BF)
        vc[i] = torch.randn((1, ps, d), generator=g, device=cuda_device).to(BF)
    q = torch.randn((70, 2, d), generator=g, device=cuda_device).to(BF)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    o, lse = fa.fa_fwd_paged(q, kc, vc, i32([ids]), i32([0, 70]), i32([500]), with_lse=True)
    ref.check_fwd_paged(q, kc, vc, [ids], [500], [70], o, lse, "far pages")


def test_many_rows_far_offsets(cuda_device):
    """o and q past 2^31 bytes: the last sequence of many tokens."""
    T, H, d = 70_000, 128, 128
    q = torch.zeros(T, H, d, dtype=BF, device=cuda_device)
    b = Batch(cuda_device, H, 1, d, 64, [(30, 5)])
    q[-5:] = b.q
    cu = torch.tensor([T - 5, T], dtype=torch.int32, device=cuda_device)
    o, lse = fa.fa_fwd_paged(q, b.kc, b.vc, b.table, cu, b.len_t, with_lse=True)
    b.check(o[-5:], lse[-5:], "far rows")


def test_finite_scale_default(cuda_device):
    b = Batch(cuda_device, 4, 2, 64, 16, [(33, 5)])
    assert torch.equal(b.run()[0], b.run(scale=1 / math.sqrt(64))[0])


def test_two_streams_at_once(cuda_device):
    """Calls of both head dimensions on two streams at the same time, each with the allocator's workspace."""
    a = Batch(cuda_device, 8, 2, 128, 16, MIXED + [(3000, 40)], seed=2)
    b = Batch(cuda_device, 8, 2, 64, 16, MIXED + [(2000, 400)], seed=3)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(25):
        got.append((a.run(stream=streams[0]), b.run(stream=streams[1])))
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK
    for pair in got:
        for x, y in zip(pair, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_back_to_back_behind_the_append(cuda_device):
    """Each launch may start before the one in front of it has ended: new keys, then the attention that reads them, many layers
    without a pause, against the same with a synchronisation between all calls."""
    d, ps, Hkv = 128, 16, 2
    b = Batch(cuda_device, 8, Hkv, d, ps, [(300, 60), (0, 33), (511, 1), (40, 2)])
    slots = torch.cat([torch.as_tensor(np.asarray(t, dtype=np.int64))[torch.arange(n - m, n) // ps] * ps + torch.arange(n - m, n) % ps
                       for t, n, m in zip(b.tables, b.lens, b.news)]).to(cuda_device)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(8)
    layers = [tuple(torch.randn((b.T, Hkv, d), generator=g, device=cuda_device).to(BF) for _ in range(2)) for _ in range(12)]
    results = []
    for pause in (True, False):
        out = []
        for k, v in layers:
            fa.fa_paged_append(k, v, b.kc, b.vc, slots)
            if pause:
                torch.cuda.synchronize()
            out.append(b.run())
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append(out)
    for x, y in zip(*results):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
