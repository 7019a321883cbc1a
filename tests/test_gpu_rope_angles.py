"""The angles of pa_rope_append: small ones to fp32's relative accuracy, and those of large
frequencies and far positions within the stated distance of the exact ones."""
import decimal
import math

import pytest
import torch

import paged_kv_cache_335_b200 as pa
from tests import plain_forms as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TAU = decimal.Decimal("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256")


def _sines(freq, pos):
    """sin and cos of every position x frequency as the kernel makes them: rows (0, 1) turn to
    (-sin, cos)."""
    t, half = len(pos), len(freq)
    q = torch.zeros((t, 1, 128), device=DEV)
    q[..., half:2 * half] = 1.0
    k, out = q.clone(), torch.empty_like(q)
    kc, vc = (torch.zeros((t // 16 + 1, 1, 16, 128), device=DEV) for _ in range(2))
    pa.pa_rope_append(out, q, k, k, torch.tensor([pos], dtype=torch.int32, device=DEV),
                      torch.arange(t, device=DEV), kc, vc, pa.rope_desc(2 * half, inv_freq=freq))
    pa.pa_sync_check()
    return -out[:, 0, :half].double().cpu(), out[:, 0, half:2 * half].double().cpu()


def _angle(p, f):
    """position x frequency modulo a turn, nearest to 0, in radians (a double of its own size)."""
    with decimal.localcontext() as c:
        c.prec = 80
        a = (decimal.Decimal(p) * decimal.Decimal(f)) % TAU
        if a > TAU / 2:
            a -= TAU
        if a < -TAU / 2:
            a += TAU
        return float(a)


@pytest.mark.parametrize("sign", [1, -1])
def test_small_angles_keep_their_relative_accuracy(sign):
    freq = [sign * 10.0 ** (-9 + 0.5 * i) for i in range(8)]
    pos = [1, -1, 2, 3, 7, -11, 20]
    sin, cos = _sines(freq, pos)
    for i, p in enumerate(pos):
        for j, f in enumerate(freq):
            a = _angle(p, f)
            # the angle rounded to fp32 (1 step of EPS32), the sine to 2 units (4), the multiplier (1), the
            # sum with 0 x cosine (1); and the fixed-point error of the angle
            tol = 7 * P.EPS32 * abs(math.sin(a)) + abs(p) * (1 + abs(f)) * 2.0 ** -65 * 2 * math.pi
            assert abs(float(sin[i, j]) - math.sin(a)) <= tol, (p, f, float(sin[i, j]), math.sin(a))
            assert abs(float(cos[i, j]) - math.cos(a)) <= 7 * P.EPS32


def test_far_positions_and_large_frequencies():
    freq = [1.0, -1.0, 6.5, 1e3, -123456.75, 1e6, 0.9999999, 1e-3]
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 99991, -1, 0, 65537]
    sin, cos = _sines(freq, pos)
    for i, p in enumerate(pos):
        for j, f in enumerate(freq):
            a = _angle(p, f)
            # half-turns rounded to fp32 (pi EPS32 radians), the functions' 4 and the products' 2
            # EPS32; the fixed-point error
            tol = (math.pi + 6) * P.EPS32 + abs(p) * (1 + abs(f)) * 2.0 ** -65 * 2 * math.pi
            assert abs(float(sin[i, j]) - math.sin(a)) <= tol, (p, f)
            assert abs(float(cos[i, j]) - math.cos(a)) <= tol, (p, f)
