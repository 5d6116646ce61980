"""How exact the paged decode's products are: o against float64 within a bound that leaves no room for P in 16 bits.

The bound counts, with u = 2^-24 and S = sum p |v| of a row:
  scores     a matrix instruction adds 16 products and the sum before it with at most 17 truncations of one step of the
             largest, so d products are off by at most 2 d u sum |q_i k_i|, times |scale|; 4 u more for the scaling: ds
  P          ex2.approx and its argument's rounding 2^-20; scores 2 ds (numerator and denominator); P = hi + lo + rest with
             hi P cut off after 8 bits, lo the nearest bf16 to what hi leaves (less than 2^-7 P), so |rest| <= 2^-15 P
  P V        2 n u S for the sums as above, both terms; 2^-19 S for the joined states' weights (a few ex2.approx and products)
  output     2^-8 |o|, the only rounding to 16 bits
With P rounded to bf16 once, |rest| would be 2^-8 P: elements of o near zero then pass the bound by several times.
"""
import math

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa
import paged_ref as ref

pytestmark = pytest.mark.gpu


def _bounded(q, k, v, scale, o, name):
    n, d = k.shape
    u = 2.0 ** -24
    ro, _, _, _ = ref.attend(q, k, v, scale)
    s = (k @ q) * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    ds = (2 * d + 4) * u * abs(scale) * (np.abs(k) @ np.abs(q)).max()
    lim = (2.0 ** -15 + 2 * ds + 2.0 ** -19 + 2.0 ** -19 + 2 * n * u) * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(ro)
    err = np.abs(o - ro)
    assert (err <= lim).all(), f"{name}: {(err > lim).sum()} of {d} outside, worst {(err / lim).max():.2f} of the bound"
    return (err / lim).max()


def _check(dev, lens, H, Hkv, d, ps, room, seed, prefix_len=0):
    tables, prefix, total = ref.deal_pages(lens, ps, seed, extra=-(-prefix_len // ps))
    kc, vc = ref.paged_cache(total, Hkv, ps, d, dev, seed + 1)
    g = torch.Generator(device=dev)
    g.manual_seed(seed + 2)
    q = (torch.randn((len(lens), H, d), generator=g, device=dev) * 0.7).to(torch.bfloat16)
    table = ref.page_table(tables, dev, max(max(map(len, tables)), -(-room // ps)))
    lens_t = torch.as_tensor(np.asarray(lens, np.int32), device=dev)
    pre = torch.as_tensor(np.asarray(prefix, np.int32), device=dev)
    o, _ = fa.fa_decode_paged_prefix(q, kc, vc, pre, prefix_len, table, lens_t)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK
    qf, of, G, worst = ref.f64(q), ref.f64(o), H // Hkv, 0.0
    for b in sorted({0, 1, len(lens) // 2, len(lens) - 1}):
        for hk in range(Hkv):
            k = ref.sequence_rows(kc, tables[b], lens[b], hk)
            v = ref.sequence_rows(vc, tables[b], lens[b], hk)
            if prefix_len:
                k = np.concatenate((ref.sequence_rows(kc, prefix, prefix_len, hk), k))
                v = np.concatenate((ref.sequence_rows(vc, prefix, prefix_len, hk), v))
            for h in range(hk * G, (hk + 1) * G):
                worst = max(worst, _bounded(qf[b, h], k, v, 1 / math.sqrt(d), of[b, h], f"sequence {b} head {h}"))
    print(f"[accuracy] d{d} H{H}/{Hkv} P{prefix_len} room {room}: worst {worst:.2f} of the bound")


@pytest.mark.parametrize("room", [0, 40_000], ids=["clusters", "ranges"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (12, 1), (33, 1)], ids=str)
def test_paged_decode_keeps_p(cuda_device, room, d, H, Hkv):
    """Groups of every tile width; sequences of a few keys (P's rounding shows most) to many tiles."""
    _check(cuda_device, [3, 2, 9, 40, 777], H, Hkv, d, 16, room, 4000 + d + H)


@pytest.mark.parametrize("room", [0, 40_000], ids=["clusters", "ranges"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,ps,prefix_len", [(3, 16, 5), (3, 5, 150), (70, 16, 333), (70, 64, 1024), (70, 24, 128)], ids=str)
def test_shared_prefix_keeps_p(cuda_device, room, d, B, ps, prefix_len):
    """Both widths of the prefix's query tiles (B * 4 rows a head), whole and ragged tiles, gathered pages, several splits."""
    _check(cuda_device, [b % 7 for b in range(B)], 8, 2, d, ps, room, 4100 + d + B, prefix_len)


@pytest.mark.parametrize("room", [0, 40_000], ids=["clusters", "ranges"])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_stay_infinite(cuda_device, room, d):
    """An infinite value that a row sees gives that infinity in its dimension, as the formula does, in the key of largest P
    (P = 1: a term of it that were zero would give NaN) as in the others; the other dimensions are as they were."""
    for prefix_len in (0, 90):
        lens = [1, 40, 100]
        tables, prefix, total = ref.deal_pages(lens, 16, 4300, extra=-(-prefix_len // 16))
        kc, vc = ref.paged_cache(total, 2, 16, d, cuda_device, 4301)
        q = ref.paged_cache(1, 3, 4, d, cuda_device, 4302)[0][0]
        table = ref.page_table(tables, cuda_device, max(7, -(-room // 16)))
        lens_t = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
        pre = torch.as_tensor(np.asarray(prefix, np.int32), device=cuda_device)

        def run():
            o, _ = fa.fa_decode_paged_prefix(q, kc, vc, pre, prefix_len, table, lens_t)
            torch.cuda.synchronize()
            assert fa.fa_check_device_error() == fa.FA_OK
            return o

        clean = run()
        want = clean.clone()
        for b, n in enumerate(lens):
            for i in range(n):  # every key in a dimension of its own
                vc[int(tables[b][i // 16]), 1, i % 16, i % (d - 1)] = -math.inf if i % (d - 1) % 2 else math.inf
            at = torch.arange(min(n, d - 1), device=cuda_device)
            want[b][2:, at] = torch.where(at % 2 == 1, -math.inf, math.inf).to(want.dtype)
        if prefix_len:
            vc[int(prefix[-1]), 0, (prefix_len - 1) % 16, d - 1] = math.inf
            want[:, :2, d - 1] = math.inf
        o = run()
        assert torch.equal(o, want)
