"""The rotation's sines and cosines against exact angles, within a bound derived from the kernel's own steps (u = 2^-24):

  frequency  F, the fraction f / (2 pi) of a turn: the constant and the product round in double, 2^-53 each of f / (2 pi); a
             negative f's fraction is rounded once more, by at most 2^-54 turns.  Times the position:
             |pos| (|f| 2^-52 + (f < 0) 2 pi 2^-54) rad
  phase      pos * F modulo a turn is exact in 64-bit integers; its lower 32 bits are cut off: 2 pi 2^-32 = 1.5e-9 rad
  argument   x, the rest to the nearest quarter turn, |x| <= pi / 4: to fp32, times an fp32 constant, rounded: 3 u |x|, so
             with the phase dx <= 1.42e-7
  sine       dx cos x; x^11 / 11! = 1.8e-9; the last addition u sin x, the terms before it 5 u x^3 / 6: below 1.7e-7
  cosine     dx sin x; x^12 / 12! = 1.2e-10; the last addition u / 2, the terms before it 3 u x^2 / 2: below 1.9e-7

Pairs (1, 0) turn into (cos, sin) with nothing added: the products are exact and the sums have a zero in them."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_forward_05_gb300 as fa

pytestmark = pytest.mark.gpu

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
POLY = 1.9e-7


def _exact(pos, f):
    turns = Fraction(f) * pos / (2 * PI)
    a = float((turns - round(turns)) * 2 * PI)  # within half a turn: nothing is lost
    return math.cos(a), math.sin(a)


FREQS = {"usual": [10000.0 ** (-i / 32) for i in range(32)],
         "above one": [7.5, 2 * math.pi, 100.25, 1e4, 3.0, 1.0, 33.3, 1e6],
         "negative": [-0.3, -1.0, -1e-9, -100.25, -2.0 ** -30, -7.5, -1e4, -0.999],
         "tiny": [1e-9, 2.0 ** -40, 0.0, 1e-5, 3e-7, 2.0 ** -62, 1e-3, 1e-300]}


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("heads", [1, 5], ids=["one head", "several"])
@pytest.mark.parametrize("which", FREQS)
def test_sines_and_cosines(cuda_device, which, heads, inverse):
    freqs = FREQS[which]
    rng = np.random.default_rng(6000)
    pos = [0, 1, -1, 2, 17, 1000, 65_537, 999_999, 999_999_937, 2 ** 31 - 1, -2 ** 31, -12_345_678]
    pos += rng.integers(-2 ** 31, 2 ** 31, 60).tolist() + rng.integers(-100_000, 100_000, 60).tolist()
    n, N = len(freqs), len(pos)
    q = torch.zeros(1, heads, N, 64, device=cuda_device)
    q[..., :n] = 1.0
    call = fa.fa_rope_bwd if inverse else fa.fa_rope
    y, _ = call(q, None, torch.tensor(pos, dtype=torch.int32, device=cuda_device),
                torch.tensor(freqs, dtype=torch.float64, device=cuda_device))
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK
    got = y.double().cpu().numpy()[0]
    assert (got[1:] == got[:1]).all()
    worst = 0.0
    for t, p in enumerate(pos):
        for i, f in enumerate(freqs):
            c, s = _exact(p, f)
            lim = POLY + abs(p) * (abs(f) * 2.0 ** -52 + (f < 0) * 2 * math.pi * 2.0 ** -54)
            err = max(abs(got[0, t, i] - c), abs(got[0, t, n + i] - (-s if inverse else s)))
            assert err <= lim, f"pos {p} f {f}: off by {err:.3e}, bound {lim:.3e}"
            worst = max(worst, err / lim)
    print(f"[angles] {which} heads {heads}: worst {worst:.2f} of the bound")


@pytest.mark.parametrize("pos", [1, 4095, 1_000_000])
def test_near_positions_keep_the_angle(cuda_device, pos):
    """Up to a million positions the frequencies' rounding is far below the sine's own error: 2.3e-10 rad at f = 1."""
    freqs = FREQS["usual"]
    q = torch.zeros(1, 4, 1, 64, device=cuda_device)
    q[..., :32] = 1.0
    y, _ = fa.fa_rope(q, None, torch.tensor([pos], dtype=torch.int32, device=cuda_device),
                      torch.tensor(freqs, dtype=torch.float64, device=cuda_device))
    got = y.double().cpu().numpy()[0, 0, 0]
    for i, f in enumerate(freqs):
        c, s = _exact(pos, f)
        assert abs(got[i] - c) <= POLY + 1e-9 and abs(got[32 + i] - s) <= POLY + 1e-9
