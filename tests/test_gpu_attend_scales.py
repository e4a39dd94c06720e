"""attend_fp8 where the V scales of a request's blocks lie far apart.

A row's result depends on the blocks that it sees alone, and a block of a negligible weight takes no bits from the others:
the bound here counts the weights (exponential times V scale) of the positions that a row sees, nothing else.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
T = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device; the CUDA path has no fallback"
    pa.build()
    pa.library()
    yield
    pa.check_error()


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def attend(q, kc, vc, ks, vs, tables, lens, off, scale, dtype):
    """(out, bound), float64.  The bound, with weights w = p * (V scale) and A = sum p |v| of an element: half a step of the
    output; P in f16, half a step 2^-11 of A, and where it is subnormal 2^-25 of the largest weight that the row sees, for
    every code; scores from float32 sums of d <= 128 products, each off by 2^-23 of the largest sum |q k| S, which moves
    p by twice that; L / 16 + 16 float32 sums of A; exponentials below 2^-110 may count for nothing."""
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    hq, hkv, bs = q.shape[1], kc.shape[1], kc.shape[2]
    g = hq // hkv
    info = torch.finfo(dtype)
    for b in range(len(lens)):
        lo, hi, L = int(off[b]), int(off[b + 1]), int(lens[b])
        for h in range(hkv):
            k, v = ref.gather(kc, ks, tables[b], L, h), ref.gather(vc, vs, tables[b], L, h)
            code = np.abs(ref.gather(vc, np.ones_like(vs), tables[b], L, h))
            sv = vs.astype(np.float64)[np.asarray(tables[b])[np.arange(L) // bs], h]
            for t in range(hi - lo):
                seen = L - (hi - lo) + t + 1
                if seen <= 0:
                    continue
                rows = q[lo + t, h * g:(h + 1) * g]
                s = scale * rows @ k[:seen].T
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                o, mass = p @ v[:seen], p @ np.abs(v[:seen])
                big = (abs(scale) * np.abs(rows) @ np.abs(k[:seen]).T).max(1, keepdims=True)
                top = (p * sv[:seen]).max(1, keepdims=True)
                out[lo + t, h * g:(h + 1) * g] = o
                bound[lo + t, h * g:(h + 1) * g] = (
                    info.eps / 2 * np.abs(o) * 1.01 + mass * (2.0 ** -11 + 2 * big * 128 * 2.0 ** -23 + (L / 16 + 16) * 2.0 ** -23)
                    + 2.0 ** -25 * top * code[:seen].sum(0) + 2.0 ** -110 * (sv[:seen, None] * code[:seen]).sum(0)
                    + info.smallest_normal * info.eps / 2)
    return out, bound


def check(got, want, bound, dtype):
    got = f64(got)
    with np.errstate(invalid="ignore"):
        wrong = ~(np.abs(got - want) <= bound)
    if dtype == torch.float16:  # outputs past f16's range (from 65520 on) are infinite
        wrong &= ~((got == np.inf) & (want + bound >= 65520)) & ~((got == -np.inf) & (want - bound <= -65520))
    assert not wrong.any(), (int(wrong.sum()), np.argwhere(wrong)[:4].tolist(), got[wrong][:4], want[wrong][:4], bound[wrong][:4])


def make(seed, old, new, hq, hkv, d, bs, dtype, q_mult=1.0):
    rng = np.random.default_rng(seed)
    kc, vc, ks, vs, tables, lens = ref.paged(rng, np.array(old) + new, hkv, d, bs)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy((rng.standard_normal((off[-1], hq, d)) * q_mult).astype(np.float32)).to(T[dtype]).cuda()
    return rng, q, kc, vc, ks, vs, tables, lens, off


def run(q, kc, vc, ks, vs, tables, lens, off, **kw):
    out = pa.attend_fp8(q, up(kc), up(vc), up(ks), up(vs), up(tables), up(lens), up(off), **kw)
    pa.check_error()
    return out


@pytest.mark.parametrize("ratio", [1e4, 1e6, 1e8, 2.0 ** 40, 1e30])
@pytest.mark.parametrize("hq", [2, 16])  # 60 rows of a kv head: one row tile; 480: pairs of them
@pytest.mark.parametrize("dtype,d,bs", [("bf16", 128, 16), ("f16", 64, 32), ("f16", 128, 32), ("bf16", 64, 32), ("bf16", 64, 16)])
def test_a_later_blocks_v_scale_leaves_earlier_rows_as_they_are(ratio, hq, dtype, d, bs):
    old, new = [0, 70, 130, 3], [60, 60, 60, 60]
    _, q, kc, vc, ks, vs, tables, lens, off = make(1, old, new, hq, 2, d, bs, dtype)
    plain = f64(run(q, kc, vc, ks, vs, tables, lens, off))
    high = vs.copy()
    last = [(n - 1) // bs for n in lens]
    for b, j in enumerate(last):
        high[tables[b, j]] *= ratio
    got = run(q, kc, vc, ks, high, tables, lens, off)
    want, bound = attend(f64(q), kc, vc, ks, high, tables, lens, off, d ** -0.5, T[dtype])
    check(got, want, bound, T[dtype])
    for b, j in enumerate(last):  # rows before that block: as with its ordinary scale
        rows = slice(off[b], off[b] + max(0, j * bs - old[b]))
        assert rows.stop > rows.start
        assert (np.abs(f64(got)[rows] - plain[rows]) <= 2 * bound[rows]).all()


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("dtype,d,bs,spread", [("bf16", 128, 16, 20), ("bf16", 64, 32, 60), ("f16", 64, 16, 12), ("f16", 128, 32, 30)])
def test_scales_far_apart_in_sight(seed, dtype, d, bs, spread):
    """V scales over 2^spread; sharp scores, so that the weight moves from block to block, whatever their scales."""
    old, new = [0, 900, 5, 260], [150, 3, 40, 1]
    rng, q, kc, vc, ks, vs, tables, lens, off = make(seed, old, new, 8, 2, d, bs, dtype, q_mult=12.0)
    vs = np.exp2(rng.uniform(-spread, 0, vs.shape)).astype(np.float32)
    want, bound = attend(f64(q), kc, vc, ks, vs, tables, lens, off, d ** -0.5, T[dtype])
    check(run(q, kc, vc, ks, vs, tables, lens, off), want, bound, T[dtype])


@pytest.mark.parametrize("order", ["first", "middle", "last"])
@pytest.mark.parametrize("apart", [40.0, 300.0])
def test_a_large_scale_of_negligible_weight_takes_no_bits(order, apart):
    """One block in sight has a V scale 2^45 times the others' and scores so far below theirs that it does not count."""
    bs, d, L, n = 16, 128, 300, 40
    _, q, kc, vc, ks, vs, tables, lens, off = make(7, [L - n], [n], 4, 1, d, bs, "bf16", q_mult=0.1)
    q[:, :, 0] = 8.0
    ks[:] = 0.01
    at = {"first": 0, "middle": 9, "last": (L - n) // bs - 1}[order]
    kc[:, :, :, 0] = 0
    code = 0x70  # 128
    kc[tables[0, at], :, :, 0] = code | 0x80
    vs[:] = 0.01
    vs[tables[0, at]] = 0.01 * 2.0 ** 45
    scale = apart / (8.0 * 128 * 0.01)
    want, bound = attend(f64(q), kc, vc, ks, vs, tables, lens, off, scale, torch.bfloat16)
    if apart > 100:  # its weight is below 2^-380
        assert (np.abs(want) < 10).all() and (bound < 2.0 ** -6 * 10).all()
    check(run(q, kc, vc, ks, vs, tables, lens, off, scale=scale), want, bound, torch.bfloat16)


def test_blocks_of_zeros_beside_blocks_of_values():
    """What rope_append_fp8 makes of zeros has the scale 2^-100."""
    _, q, kc, vc, ks, vs, tables, lens, off = make(9, [200, 0, 77], [3, 150, 60], 4, 2, 128, 16, "bf16", q_mult=4.0)
    for b in range(3):
        for j in range(0, len(tables[b]), 2):
            if tables[b, j] >= 0:
                vc[tables[b, j]], vs[tables[b, j]] = 0, 2.0 ** -100
    want, bound = attend(f64(q), kc, vc, ks, vs, tables, lens, off, 128 ** -0.5, torch.bfloat16)
    check(run(q, kc, vc, ks, vs, tables, lens, off), want, bound, torch.bfloat16)


@pytest.mark.parametrize("new", [1, 200])
def test_parts_of_a_long_context_with_scales_far_apart(new):
    """Contexts cut into parts, some of large scales and little weight."""
    rng, q, kc, vc, ks, vs, tables, lens, off = make(11, [9000, 7000], [new, new], 4, 1, 64, 16, "bf16", q_mult=6.0)
    vs = np.exp2(rng.uniform(-30, 30, vs.shape)).astype(np.float32)
    want, bound = attend(f64(q), kc, vc, ks, vs, tables, lens, off, 0.125, torch.bfloat16)
    check(run(q, kc, vc, ks, vs, tables, lens, off), want, bound, torch.bfloat16)
