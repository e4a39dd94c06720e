"""Host-side checks of the serving-step operators (no GPU): argument validation and rotary frequencies."""
import math

import pytest
import torch

import paged_kv_cache_129_gb300 as pa

P = 1 << 30  # an aligned, never-dereferenced address; buffers below are far apart


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.library()


def spaced(n):
    return [P + (i << 28) for i in range(n)]


def check(fn, ok, changes, status):
    for i, value in changes.items():
        args = list(ok)
        args[i] = value
        assert fn(*args) == status, (i, value)


def test_advance_tables_rejects_bad_arguments(lib):
    b = spaced(10)
    #     tables, lens, new, stack, count | lens out, count out, offsets, positions, slots | seqs, width, blocks, bs, tokens
    ok = b + [4, 8, 100, 16, 64, None]
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):
        check(lib.pa_advance_tables, ok, {i: None}, 1)
        check(lib.pa_advance_tables, ok, {i: b[i] + 2}, 1)
    check(lib.pa_advance_tables, ok, {9: b[9] + 4, 10: 8193, 11: 0, 12: 0, 13: 0, 14: -1}, 1)
    check(lib.pa_advance_tables, ok, {10: -1, 11: 1 << 28}, 1)
    # overlapping buffers; lengths and count alone may be in place
    check(lib.pa_advance_tables, ok, {5: b[2], 6: b[3] + 396, 7: b[1], 8: b[9] + 8, 9: b[0]}, 1)
    check(lib.pa_advance_tables, ok, {5: b[1] + 4, 6: b[5]}, 1)


def test_rope_write_rejects_bad_arguments(lib):
    b = spaced(9)  # query_out, query, key, value, key_cache, value_cache, inv_freq, positions, slots
    ok = b + [512, 256, 256, 8, 4, 2, 128, 128, 0, 1.0, 16, 10, 2, None]
    for i in range(9):
        check(lib.pa_rope_write_kv, ok, {i: None}, 1)
        check(lib.pa_rope_write_kv, ok, {i: b[i] + 1}, 1)
    check(lib.pa_rope_write_kv, ok, {9: 511, 10: 255, 11: 255}, 1)  # token strides
    check(lib.pa_rope_write_kv, ok, {12: -1, 13: 0, 14: 0, 15: 127, 16: 130, 17: 2, 19: 0, 20: 0, 21: 3}, 1)
    check(lib.pa_rope_write_kv, ok, {16: 63}, 1)
    check(lib.pa_rope_write_kv, ok, {18: float("inf")}, 1)
    check(lib.pa_rope_write_kv, ok, {0: b[1] + 64, 1: b[0] - 64, 2: b[0] + 128, 3: b[0] - 2}, 1)  # overlaps
    strided = list(ok)
    strided[9], strided[0] = 1024, strided[1]
    assert lib.pa_rope_write_kv(*strided) == 1  # in place with strided queries
    empty = list(ok)
    empty[12] = 0
    assert lib.pa_rope_write_kv(*empty) == 0
    wide = list(ok)
    wide[15], wide[9], wide[10], wide[11] = 514, 4 * 514, 2 * 514, 2 * 514
    assert lib.pa_rope_write_kv(*wide) == 2


def test_rope_append_rejects_bad_arguments(lib):
    b = spaced(12)  # query_out, query, key, value, caches, scales, inv_freq, tables, lens, offsets
    ok = b + [512, 256, 256, 3, 8, 4, 2, 128, 128, 0, 1.0, 16, 8, 10, 2, None]
    for i in (0, 1, 2, 3, 4, 6, 7, 8, 9, 10, 11):
        check(lib.pa_rope_append_fp8, ok, {i: None}, 1)
        check(lib.pa_rope_append_fp8, ok, {i: b[i] + 1}, 1)
    check(lib.pa_rope_append_fp8, ok, {5: b[5] + 4}, 1)  # (a NULL value cache means records)
    check(lib.pa_rope_append_fp8, ok, {15: -1, 16: -1, 17: 0, 18: 0, 20: 130, 21: 2, 24: 0, 25: 0, 26: 3}, 1)
    check(lib.pa_rope_append_fp8, ok, {20: 126, 23: 8}, 2)
    d96 = list(ok)
    d96[19], d96[20] = 96, 96
    assert lib.pa_rope_append_fp8(*d96) == 2
    for i in (15, 16):
        empty = list(ok)
        empty[i] = 0
        assert lib.pa_rope_append_fp8(*empty) == 0


def test_attend_rejects_bad_arguments(lib):
    b = spaced(9)  # out, query, caches, scales, tables, lens, offsets
    ok = b + [3, 8, 4, 2, 128, 16, 8, 10, 0.1, 2, None, 0, None]
    for i in (0, 1, 2, 4, 5, 6, 7, 8):
        check(lib.pa_attend_fp8, ok, {i: None}, 1)
        check(lib.pa_attend_fp8, ok, {i: b[i] + 2}, 1)
    check(lib.pa_attend_fp8, ok, {3: b[3] + 8, 0: b[1] + 16}, 1)
    check(lib.pa_attend_fp8, ok, {9: -1, 10: -1, 11: 3, 12: 0, 15: 0, 16: 0, 17: float("nan")}, 1)
    check(lib.pa_attend_fp8, ok, {16: 1 << 27, 15: 1 << 28, 10: 1 << 29}, 1)
    check(lib.pa_attend_fp8, ok, {13: 256, 14: 8, 18: 0, 9: 8193}, 2)
    for i in (9, 10):
        empty = list(ok)
        empty[i] = 0
        assert lib.pa_attend_fp8(*empty) == 0


def test_python_checks_refuse_host_tensors_and_shapes(lib):
    x = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        pa.advance_tables(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                          torch.zeros(1, dtype=torch.int32), 16, 4)
    with pytest.raises(ValueError):
        pa.rope_write_kv(x, x, x, torch.zeros(1, 2, 16, 64), torch.zeros(1, 2, 16, 64), torch.zeros(32, dtype=torch.float64),
                         torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64))
    codes, scale = torch.zeros(1, 2, 16, 64, dtype=torch.uint8), torch.zeros(1, 2)
    with pytest.raises(ValueError):
        pa.rope_append_fp8(x, x, x, codes, codes, scale, scale, None, torch.zeros(1, 1, dtype=torch.int32),
                           torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        pa.attend_fp8(x.half(), codes, codes, scale, scale, torch.zeros(1, 1, dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "ramp"])
def test_rope_frequencies(scaling):
    r, base, factor, ctx = 64, 10000.0, 4.0, 2048
    got = pa.rope_frequencies(r, base, scaling, factor, context=ctx, low=2.0, high=20.0)
    assert got.dtype == torch.float64 and got.shape == (r // 2,)
    for i in range(r // 2):
        f = base ** (-2 * i / r)
        if scaling == "linear":
            f /= factor
        elif scaling == "base":
            f = (base * factor ** (r / (r - 2))) ** (-2 * i / r)
        elif scaling == "ramp":
            keep = min(1.0, max(0.0, (ctx * f / (2 * math.pi) - 2.0) / 18.0))
            f = f * keep + f / factor * (1 - keep)
        assert abs(float(got[i]) - f) <= 1e-14 * f


def test_rope_frequencies_refuses_bad_arguments():
    for bad in ({"rotary_dim": 3}, {"rotary_dim": 0}, {"rotary_dim": 8, "scaling": "other"}, {"rotary_dim": 8, "factor": 0.0},
                {"rotary_dim": 2, "scaling": "base"}, {"rotary_dim": 8, "scaling": "ramp"}):
        with pytest.raises(ValueError):
            pa.rope_frequencies(**bad)
