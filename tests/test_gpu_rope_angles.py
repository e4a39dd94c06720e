"""Rotary angles of positions up to the ends of int32, against whole-number arithmetic.

A head holds (1, 0) in every pair, so that the rotated pair is (cos, sin) of the angle itself.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa

pytestmark = pytest.mark.gpu
BITS = 320
# 2^-28 turns of angle (the float32 that goes to sincospi, and 2^-32 for the fixed point) and two units in the last place
# of sincospi below 1
SLACK = 2 * np.pi * (2.0 ** -28 + 2.0 ** -32) + 2 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device; the CUDA path has no fallback"
    pa.build()
    pa.library()
    yield
    pa.check_error()


def pi():
    """pi * 2^BITS as a whole number: 16 atan(1 / 5) - 4 atan(1 / 239), with 32 bits to spare."""
    one = 1 << (BITS + 32)

    def atan_of_inverse(x):
        total, power, n = 0, one // x, 1
        while power:
            total += power // n if n % 4 == 1 else -(power // n)
            power //= x * x
            n += 2
        return total

    return (16 * atan_of_inverse(5) - 4 * atan_of_inverse(239)) >> 32


def turns(inv_freq, pos):
    """The angle pos * inv_freq in turns, without whole ones, in [-1/2, 1/2]."""
    a = Fraction(float(inv_freq)) * int(pos) / (2 * Fraction(pi(), 1 << BITS))
    a -= round(a)
    return float(a)


# frequencies whose quotient by 2 pi is far from its double, fast ones among them
FREQ = np.array([1.0, 0.75, 3.9, 5.1, 1 / 3, 0.1, 7.7, 100.3, 1e-3, 1e-9, -2.3, 12345.678])
POS = np.array([0, 1, -1, 4095, 10 ** 6, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, -2 ** 31 + 7], np.int64)


def expected():
    a = np.array([[turns(f, p) for f in FREQ] for p in POS]) * 2 * np.pi
    return np.cos(a), np.sin(a)


def check(rows):
    """rows [positions, ..., 2 * frequencies] in the half layout."""
    c, s = expected()
    got = rows.double().cpu().numpy().reshape(len(POS), -1, 2, len(FREQ))
    err = np.maximum(np.abs(got[:, :, 0] - c[:, None]), np.abs(got[:, :, 1] - s[:, None]))
    assert (err <= SLACK).all(), (err.max() / SLACK, np.argwhere(err > SLACK)[:5].tolist())


@pytest.mark.parametrize("copies", [1, 64])  # a token per CTA; four
def test_rope_write_kv_angles(copies):
    d, t = 2 * len(FREQ), len(POS)
    x = torch.zeros(t * copies, 1, d, device="cuda")
    x[..., :d // 2] = 1
    kc, vc = (torch.zeros(t * copies, 1, 1, d, device="cuda") for _ in range(2))
    slots = torch.arange(t * copies, device="cuda")
    pos = torch.from_numpy(POS.astype(np.int32)).cuda().repeat_interleave(copies)
    q = pa.rope_write_kv(x, x, x, kc, vc, torch.from_numpy(FREQ).cuda(), pos, slots)
    pa.check_error()
    check(q.view(t, copies, d))
    check(kc.view(t, copies, d))


def test_rope_append_fp8_angles():
    """Requests of one new token each, at POS's positions that a table can reach."""
    d, bs, rot = 64, 16, 2 * len(FREQ)
    pos = [p for p in POS if 0 <= p < 2 ** 21]
    width = max(pos) // bs + 1
    tables = torch.zeros(len(pos), width, dtype=torch.int32, device="cuda")
    for b, p in enumerate(pos):
        tables[b, p // bs] = b
    x = torch.zeros(len(pos), 1, d, device="cuda")
    x[..., :rot // 2] = 1
    codes = [torch.zeros(len(pos), 1, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(len(pos), 1, device="cuda") for _ in range(2)]
    lens = torch.tensor([p + 1 for p in pos], dtype=torch.int32, device="cuda")
    off = torch.arange(len(pos) + 1, dtype=torch.int32, device="cuda")
    q = pa.rope_append_fp8(x, x, x, *codes, *scales, torch.from_numpy(FREQ).cuda(), tables, lens, off)
    pa.check_error()
    c, s = expected()
    at = [list(POS).index(p) for p in pos]
    got = q[..., :rot].double().cpu().numpy().reshape(len(pos), 2, len(FREQ))
    assert (np.abs(got[:, 0] - c[at]) <= SLACK).all() and (np.abs(got[:, 1] - s[at]) <= SLACK).all()
