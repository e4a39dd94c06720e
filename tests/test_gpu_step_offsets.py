"""Offsets of runs that do not ascend, begin below zero or end past the rows: reported, and nothing outside the runs is touched."""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa

pytestmark = pytest.mark.gpu
BS, D = 16, 64


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device; the CUDA path has no fallback"
    pa.build()
    pa.library()
    yield
    pa.check_error()


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def status(call):
    call()
    with pytest.raises(pa.PAError) as e:
        pa.check_error()
    return e.value.status


# offsets, lengths, rows, requests that are served all the same (their runs are whole and the search meets them)
BAD = [
    ([0, 2, 5], [2, 3], 4, [0]),           # ends past the rows
    ([0, 2, 4, 9], [2, 2, 5], 4, [0, 1]),  # begins behind the rows
    ([-1, 2, 4], [3, 2], 4, [1]),          # begins below zero
    ([2, 1, 4], [1, 3], 4, []),            # descends
    ([50, 64, 0], [48, 3], 64, []),        # a row before the run that the search ends at
    ([40, 60, 2, 64], [28, 9, 62], 64, []),
    ([0, 4, 4, 2], [4, 0, 0], 4, [0]),
]


@pytest.mark.parametrize("off,lens,rows,served", BAD)
def test_rope_append_fp8_reports_offsets_that_are_none(off, lens, rows, served):
    if off[-1] < off[-2]:  # (a search of the offsets may miss runs that are whole)
        served = []
    b, width = len(lens), 8
    x = torch.ones(rows, 1, D, device="cuda")
    # the table's rows lie inside a larger one whose other entries are blocks of the pool too: a stray read would write to them
    blocks = (b + 2) * width
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda").view(b + 2, width)[1:-1]
    k, v = (torch.zeros(blocks, 1, BS, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((blocks, 1), 0.5, device="cuda") for _ in range(2))
    out = torch.full((rows, 1, D), 9.0, device="cuda")
    assert status(lambda: pa.rope_append_fp8(x, x, x, k, v, ks, vs, None, tables, i32(lens), i32(off), query_out=out)) == 7
    places = torch.zeros_like(k)  # of the runs that are whole
    for r in range(b):
        if 0 <= off[r] <= off[r + 1] <= rows:
            for p in range(lens[r] - off[r + 1] + off[r], lens[r]):
                places[(r + 1) * width + p // BS, 0, p % BS] = 0x7E  # 448 scales of 1 / 448
    for c in (k, v):
        assert int(((c != 0) & (places == 0)).count_nonzero()) == 0
        for r in served:
            assert torch.equal(c[(r + 1) * width:(r + 2) * width], places[(r + 1) * width:(r + 2) * width])
    for r in served:
        assert (out[off[r]:off[r + 1]] == 1.0).all()


@pytest.mark.parametrize("off,lens,rows,served", BAD)
def test_attend_fp8_reports_offsets_that_are_none(off, lens, rows, served):
    b, width = len(lens), 8
    q = torch.randn(rows, 1, D, device="cuda").half()
    tables = torch.arange(b * width, dtype=torch.int32, device="cuda").view(b, width)
    k, v = (torch.randint(0, 0x70, (b * width, 1, BS, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks = torch.full((b * width, 1), 0.01, device="cuda")
    out = torch.full_like(q, 9.0)
    assert status(lambda: pa.attend_fp8(q, k, v, ks, ks, tables, i32(lens), i32(off), out=out)) == 7
    seen = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for r in served:  # as the request alone
        lo, hi = off[r], off[r + 1]
        seen[lo:hi] = True
        alone = pa.attend_fp8(q[lo:hi].contiguous(), k, v, ks, ks, tables[r:r + 1], i32(lens[r:r + 1]), i32([0, hi - lo]))
        pa.check_error()
        assert torch.allclose(out[lo:hi].float(), alone.float(), rtol=2 ** -9, atol=2 ** -9 * float(alone.abs().max()))
    if served:
        assert (out[~seen] == 9.0).all()
    assert torch.isfinite(out).all()
