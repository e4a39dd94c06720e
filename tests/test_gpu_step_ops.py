"""GPU parity of the serving-step operators against float64 forms (step_reference.py) and the host block pool.

advance_tables: equal to the pool's release and append; refused steps change nothing.  rope_write_kv and rope_append_fp8:
within float32 arithmetic and one rounding; scales and codes of values that need no rotation bit for bit.  attend_fp8:
within the bound that step_reference.attend derives.  All four as a step: captured, replayed, and on a side stream.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


def status(call):
    """The error that a call leaves in the device error word."""
    call()
    with pytest.raises(pa.PAError) as e:
        pa.check_error()
    return e.value.status


# ---- tables --------------------------------------------------------------------------------

def host_step(tables, lens, new, stack, free, bs):
    """One token after the other, one id after the other."""
    tables, lens, stack = tables.copy(), lens.copy(), list(stack[:free])
    for b in np.flatnonzero(new < 0):
        stack += list(tables[b, :(lens[b] + bs - 1) // bs])
        lens[b] = 0
    pos, slots, off = [], [], [0]
    for b in range(len(lens)):
        for p in range(lens[b], lens[b] + max(new[b], 0)):
            if p % bs == 0:
                tables[b, p // bs] = stack.pop()
            pos.append(p)
            slots.append(int(tables[b, p // bs]) * bs + p % bs)
        lens[b] += max(new[b], 0)
        off.append(len(pos))
    return tables, lens, stack, off, pos, slots


@pytest.mark.parametrize("b,bs,lo,hi,pad,in_place", [
    (1, 16, 1, 1, 0, False), (5, 16, -1, 40, 7, True), (64, 16, 1, 1, 0, True), (300, 32, -1, 70, 129, False),
    (3, 1, 0, 9, 2, True), (2, 7, 0, 5000, 0, False), (1500, 16, -1, 3, 0, True), (8192, 16, -1, 1, 4, False),
    (0, 16, 0, 0, 5, False)])
def test_advance_tables_pops_what_the_pool_would(b, bs, lo, hi, pad, in_place):
    rng = np.random.default_rng(b * 31 + bs)
    lens = rng.integers(0, 3 * bs + 2, b).astype(np.int32)
    new = rng.integers(lo, hi + 1, b).astype(np.int32)
    width = int(max([(int(x) + max(int(n), 0) + bs - 1) // bs for x, n in zip(lens, new)], default=0)) + 2
    count = (lens + bs - 1) // bs
    nb = int(count.sum()) + int(np.maximum(new, 0).sum()) // bs + b + 4
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((b, width), -7, np.int32)
    at = 0
    for i, n in enumerate(count):
        tables[i, :n] = perm[at:at + n]
        at += n
    stack = np.full(nb, -9, np.int32)
    stack[:nb - at] = perm[at:]
    want = host_step(tables, lens, new, stack, nb - at, bs)
    tok = len(want[4])
    dt, dl, df, dn = up(tables), up(lens), up(stack), torch.tensor([nb - at], dtype=torch.int32, device="cuda")
    out = None
    if in_place:
        i32 = {"dtype": torch.int32, "device": "cuda"}
        out = (dl, dn, torch.empty(b + 1, **i32), torch.empty(tok + pad, **i32),
               torch.empty(tok + pad, dtype=torch.int64, device="cuda"))
    got = pa.advance_tables(dt, dl, up(new), df, dn, bs, tok + pad, out=out)
    pa.check_error()
    assert np.array_equal(dt.cpu().numpy(), want[0])
    assert np.array_equal(got.context_lens.cpu().numpy(), want[1])
    n = int(got.num_free)
    assert n == len(want[2]) and df[:n].cpu().tolist() == want[2]
    assert got.q_offsets.cpu().tolist() == want[3]
    assert got.positions.cpu().tolist() == want[4] + [0] * pad
    assert got.slot_mapping.cpu().tolist() == want[5] + [-1] * pad


def test_advance_tables_matches_the_host_pool_over_many_steps():
    rng = np.random.default_rng(5)
    bs, b, nb, width = 16, 9, 90, 12
    order = rng.permutation(nb).tolist()
    pool = pa.BlockPool(nb, bs, order)
    ids = [pool.create() for _ in range(b)]
    i32 = {"dtype": torch.int32, "device": "cuda"}
    tables, lens = torch.full((b, width), -1, **i32), torch.zeros(b, **i32)
    stack, free = torch.tensor(order, **i32), torch.tensor([nb], **i32)
    for _ in range(25):
        have = lens.cpu().numpy()
        new = np.minimum(rng.integers(-1, 30, b), width * bs - have).astype(np.int32)
        slots = []
        for i in np.flatnonzero(new < 0):
            pool.release(ids[i])
            ids[i] = pool.create()
        if pool.blocks_needed(ids, np.maximum(new, 0)) > pool.num_free():
            new[new >= 0] = 0
        for i in range(b):
            slots += [pool.append(ids[i])[0] for _ in range(max(new[i], 0))]
        got = pa.advance_tables(tables, lens, up(new), stack, free, bs, len(slots) + 3)
        lens, free = got.context_lens, got.num_free
        assert got.slot_mapping.cpu().tolist() == slots + [-1] * 3
        want, want_lens = pool.block_tables(ids, width)
        assert np.array_equal(lens.cpu().numpy(), want_lens)
        mine = tables.cpu().numpy()
        assert all(np.array_equal(mine[i, :(n + bs - 1) // bs], want[i, :(n + bs - 1) // bs]) for i, n in enumerate(want_lens))
        assert stack[:int(free)].cpu().tolist() == pool.free_list()
    pa.check_error()


@pytest.mark.parametrize("what,code", [("pool", 4), ("rows", 7), ("width", 7), ("negative", 7), ("stack", 5), ("table", 5),
                                       ("tail", 5), ("count", 5)])
def test_advance_tables_refuses_a_step_as_a_whole(what, code):
    bs, width, nb = 16, 4, 12
    tables = np.array([[3, -1, -1, -1], [4, 5, -1, -1], [6, -1, -1, -1]], np.int32)
    lens, new = np.array([10, 32, 16], np.int32), np.array([20, 3, -1], np.int32)
    stack, free, rows = np.array([0, 1, 2] + [-1] * 9, np.int32), 3, 23
    if what == "pool":
        new[1] = 32
        new[0], rows, free = 54, 86, 1  # 3 + 2 blocks, 1 + 1 free
    elif what == "rows":
        rows = 22
    elif what == "width":
        new[0], rows = 55, 60
    elif what == "negative":
        lens[2] = -1
    elif what == "stack":
        stack[2], new[2] = 12, 0
    elif what == "table":
        tables[2, 0] = -1
    elif what == "tail":
        tables[0, 0] = 99
    else:
        free = 13
    dt, dl, df, dn = up(tables), up(lens), up(stack), torch.tensor([free], dtype=torch.int32, device="cuda")
    got = []
    assert status(lambda: got.append(pa.advance_tables(dt, dl, up(new), df, dn, bs, rows))) == code
    got = got[0]
    assert np.array_equal(dt.cpu().numpy(), tables) and np.array_equal(got.context_lens.cpu().numpy(), lens)
    assert int(got.num_free) == free and df[:min(free, 3)].cpu().tolist() == stack[:min(free, 3)].tolist()
    assert got.q_offsets.cpu().tolist() == [0] * 4 and got.slot_mapping.cpu().tolist() == [-1] * rows


# ---- rotary write --------------------------------------------------------------------------

def qkv(rng, t, hq, hkv, d, dtype, fused, mult=1.0):
    x = torch.from_numpy((rng.standard_normal((t, (hq + 2 * hkv) * d)) * mult).astype(np.float32)).to(T[dtype]).cuda()
    q, k, v = x.split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
    return (q, k, v) if fused else tuple(y.contiguous() for y in (q, k, v))


def near(got, want, slack, dtype):
    err = np.abs(got - want)
    info = torch.finfo(T[dtype])  # half a step: eps / 2 relative, or that of the smallest normal number
    tol = slack + info.eps / 2 * 1.01 * np.maximum(np.abs(want), info.smallest_normal)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("t,hq,hkv,d,rot,bs,fused", [
    (1, 1, 1, 64, 64, 16, False), (5, 28, 4, 128, 128, 16, True), (67, 4, 2, 64, 16, 32, True), (33, 3, 1, 80, 20, 5, False),
    (9, 2, 2, 6, 2, 1, True), (4097, 2, 1, 128, 96, 16, True), (3, 1, 1, 512, 510, 16, False)])
def test_rope_write_kv(dtype, layout, t, hq, hkv, d, rot, bs, fused):
    rng = np.random.default_rng(t + d + rot)
    q, k, v = qkv(rng, t, hq, hkv, d, dtype, fused)
    nb = (t + bs - 1) // bs + 2
    pos = rng.integers(-1000, 1 << 20, t).astype(np.int32)
    pos[0] = 2 ** 31 - 1
    slots = rng.permutation(nb * bs)[:t].astype(np.int64)
    slots[rng.random(t) < 0.2] = -1
    inv = pa.rope_frequencies(rot, device="cuda")
    kc = torch.full((nb, hkv, bs, d), 3.0, dtype=T[dtype], device="cuda")
    vc = torch.full_like(kc, 5.0)
    out = pa.rope_write_kv(q, k, v, kc, vc, inv, up(pos), up(slots), layout=layout, factor=1.25)
    pa.check_error()
    # both float64 angles are off by p * 2^-53 * inv_freq: 2e-7 each at 2^31, as much again as the slack
    q_want, q_slack = ref.rotate(f64(q), pos, inv.cpu().numpy(), layout, 1.25)
    k_want, k_slack = ref.rotate(f64(k), pos, inv.cpu().numpy(), layout, 1.25)
    q_slack, k_slack = q_slack * 2, k_slack * 2
    near(f64(out), q_want, q_slack, dtype)
    kw, vw, sl = np.full(kc.shape, 3.0), np.full(kc.shape, 5.0), np.zeros(kc.shape)
    use = slots >= 0
    kw[slots[use] // bs, :, slots[use] % bs] = k_want[use]
    sl[slots[use] // bs, :, slots[use] % bs] = k_slack[use]
    vw[slots[use] // bs, :, slots[use] % bs] = f64(v)[use]
    near(f64(kc), kw, sl, dtype)
    assert np.array_equal(f64(vc), vw)
    assert np.array_equal(f64(out)[..., rot:], f64(q)[..., rot:])


def test_rope_write_kv_in_place_and_bad_slot():
    rng = np.random.default_rng(2)
    q, k, v = qkv(rng, 7, 4, 2, 64, "bf16", False)
    kc, vc = (torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    inv, pos = pa.rope_frequencies(64, device="cuda"), up(np.arange(7, dtype=np.int32))
    slots = np.arange(7, dtype=np.int64)
    want = pa.rope_write_kv(q, k, v, kc, vc, inv, pos, up(slots))
    kept = kc.clone()
    slots[3] = 32
    same = q.clone()
    assert status(lambda: pa.rope_write_kv(same, k, v, kc, vc, inv, pos, up(slots), query_out=same)) == 6
    assert torch.equal(same, want) and torch.equal(kc, kept)


# ---- FP8 append -------------------------------------------------------------------------------

def cache_pair(kc, vc, records):
    if records:
        return up(np.stack([kc, vc], 2)), None
    return up(kc), up(vc)


def codes_of(k, v, records):
    return (k[:, :, 0].cpu().numpy(), k[:, :, 1].cpu().numpy()) if records else (k.cpu().numpy(), v.cpu().numpy())


def expected_append(x, exact32, codes, scale, tables, lens, offsets, bs):
    """Blocks that x [T, h, d] float64 goes into: {(block, head): (first row, offset, rows, scale)} and the codes and scales
    if every step is taken in float32 (what the library does for values that need no rotation)."""
    units, codes, scale = {}, codes.copy(), scale.copy()
    for b in range(len(lens)):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        t = lo
        while t < hi:
            pos = int(lens[b]) - hi + t
            n, off, blk = min(hi - t, bs - pos % bs), pos % bs, int(tables[b, pos // bs])
            for h in range(x.shape[1]):
                a = np.abs(x[t:t + n, h])
                a = a[np.isfinite(a)].max(initial=0.0)
                held = np.float32(scale[blk, h]) if off else np.float32(0)
                s = max(held, np.float32(a) / np.float32(448), np.float32(2.0 ** -100))
                units[blk, h] = (t, off, n, s, held)
                if exact32:
                    def code(y):
                        return torch.from_numpy(y).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()

                    if off and s > held:
                        old = ref.E4M3[codes[blk, h, :off]].astype(np.float32)
                        codes[blk, h, :off] = code(old * held / s)
                    with np.errstate(over="ignore", invalid="ignore"):
                        codes[blk, h, off:off + n] = code(x[t:t + n, h].astype(np.float32) / s)
                    scale[blk, h] = s
            t += n
    return units, codes, scale


APPEND = [
    # hq, hkv, d, bs, rot, old lengths, new lengths
    (4, 2, 128, 16, 128, [0, 5, 16, 31], [1, 1, 1, 1]),
    (7, 1, 128, 16, 64, [0, 15, 40, 0, 3], [33, 0, 100, 0, 13]),
    (8, 8, 64, 32, 64, [0, 33, 1], [32, 31, 200]),
    (6, 2, 64, 16, 20, [9], [1]),
    (2, 2, 128, 32, 4, [100, 0], [60, 1000]),
    (28, 4, 128, 16, 128, [70] * 40, [3] * 40),
    (4, 4, 64, 16, 64, [13] * 700, [1, 2, 5, 0, 20, 1, 3] * 100),
]


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("records,layout", [(False, "half"), (True, "interleaved")])
def test_rope_append_fp8(case, dtype, records, layout):
    hq, hkv, d, bs, rot, old, new = case
    rng = np.random.default_rng(len(old) * 100 + d + bs)
    lens = np.array(old) + new
    kc, vc, ks, vs, tables, lens = ref.paged(rng, lens, hkv, d, bs, nan_tail=False)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t, pad = int(off[-1]), 3
    q, k, v = qkv(rng, t + pad, hq, hkv, d, dtype, True, mult=3.0)
    inv = pa.rope_frequencies(rot, device="cuda")
    dk, dv = cache_pair(kc, vc, records)
    dks, dvs = up(ks), up(vs)
    out = torch.full((t + pad, hq, d), 9.0, dtype=T[dtype], device="cuda")
    pa.rope_append_fp8(q, k, v, dk, dv, dks, dvs, inv, up(tables), up(lens), up(off), layout=layout, factor=0.75, query_out=out)
    pa.check_error()
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(old, new)])
    want, slack = ref.rotate(f64(q)[:t], pos, inv.cpu().numpy(), layout, 0.75)
    near(f64(out)[:t], want, slack, dtype)
    assert (out[t:] == 9.0).all()
    gk, gv = codes_of(dk, dv, records)
    _, want_v, want_s = expected_append(f64(v)[:t], True, vc, vs, tables, lens, off, bs)
    assert np.array_equal(gv, want_v) and np.array_equal(dvs.cpu().numpy(), want_s)
    # keys: the scale within float32 arithmetic (a pair's two elements are at most twice the block's largest), codes
    # within half a step of it
    xk, _ = ref.rotate(f64(k)[:t], pos, inv.cpu().numpy(), layout, 0.75)
    units, _, _ = expected_append(xk, False, kc, ks, tables, lens, off, bs)
    got_s = dks.cpu().numpy().astype(np.float64)
    touched = np.zeros(ks.shape, bool)
    for (blk, h), (row, o, n, s, held) in units.items():
        touched[blk, h] = True
        assert abs(got_s[blk, h] - s) <= 1.5e-6 * s
        if o:
            if got_s[blk, h] == held:
                assert np.array_equal(gk[blk, h, :o], kc[blk, h, :o])
            else:
                was = ref.E4M3[kc[blk, h, :o]] * held
                err = np.abs(ref.E4M3[gk[blk, h, :o]] * got_s[blk, h] - was)
                assert (err <= np.maximum(2.0 ** -4 * np.abs(was), 2.0 ** -10 * s) + 2e-6 * 448 * s).all()
        x = xk[row:row + n, h]
        err = np.abs(ref.E4M3[gk[blk, h, o:o + n]] * got_s[blk, h] - x)
        assert (err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) + 2e-6 * 448 * s).all()
        assert np.array_equal(gk[blk, h, o + n:], kc[blk, h, o + n:])
    assert np.array_equal(got_s[~touched], ks[~touched].astype(np.float64))
    rest = [blk for blk in range(len(kc)) if not touched[blk].any()]
    assert np.array_equal(gk[rest], kc[rest])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_append_fp8_of_views_at_odd_addresses(dtype, layout):
    """Rows that begin at any element and follow one another at an odd distance."""
    rng = np.random.default_rng(21)
    hq, hkv, d, bs, old, new = 3, 2, 64, 16, [5, 0, 30], [1, 40, 3]
    kc, vc, ks, vs, tables, lens = ref.paged(rng, np.array(old) + new, hkv, d, bs, nan_tail=False)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t, width = int(off[-1]), (hq + 2 * hkv) * d + 3
    flat = torch.from_numpy((rng.standard_normal(t * width + 1) * 3).astype(np.float32)).to(T[dtype]).cuda()
    rows = flat[1:].view(t, width)
    q, k, v = (rows[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    inv = pa.rope_frequencies(d, device="cuda")
    dk, dv, dks, dvs = up(kc), up(vc), up(ks), up(vs)
    got = pa.rope_append_fp8(q, k, v, dk, dv, dks, dvs, inv, up(tables), up(lens), up(off), layout=layout)
    pa.check_error()
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(old, new)])
    want, slack = ref.rotate(f64(q), pos, inv.cpu().numpy(), layout, 1.0)
    near(f64(got), want, slack, dtype)
    _, want_v, want_s = expected_append(f64(v), True, vc, vs, tables, lens, off, bs)
    assert np.array_equal(dv.cpu().numpy(), want_v) and np.array_equal(dvs.cpu().numpy(), want_s)
    xk, _ = ref.rotate(f64(k), pos, inv.cpu().numpy(), layout, 1.0)
    units, _, _ = expected_append(xk, False, kc, ks, tables, lens, off, bs)
    gk, gs = dk.cpu().numpy(), dks.cpu().numpy().astype(np.float64)
    for (blk, h), (row, o, n, s, held) in units.items():
        assert abs(gs[blk, h] - s) <= 1.5e-6 * s
        x = xk[row:row + n, h]
        err = np.abs(ref.E4M3[gk[blk, h, o:o + n]] * gs[blk, h] - x)
        assert (err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) + 2e-6 * 448 * s).all()


@pytest.mark.parametrize("scale", [1.0, 3.0, 0.7, 1.1e-30, 5e35])
def test_rope_append_fp8_codes_of_values_next_to_ties(scale):
    """Codes are those of the float32 quotient, at the midpoints between E4M3 values and a few float32 steps beside them too."""
    finite = ref.E4M3[:0x7F].astype(np.float64)
    mid = (finite[1:] + finite[:-1]) / 2
    d, bs, hkv = 128, 16, 1
    scale = np.float32(scale)
    x = np.zeros((bs, hkv, d), np.float32)
    base = (np.concatenate([mid, [0.0, 448.0]]).astype(np.float64) * float(scale)).astype(np.float32)
    for r in range(bs):  # row r: r - 8 steps of float32 beside them
        y = base.copy()
        y[y > 0] = (y[y > 0].view(np.int32) + (r - 8)).view(np.float32)
        x[r, 0] = np.minimum(y, np.float32(448) * scale) * np.where(np.arange(d) % 2, -1, 1)
    tables, lens, off = np.zeros((1, 1), np.int32), np.array([bs], np.int32), np.array([0, bs], np.int32)
    kc, ks = np.zeros((1, hkv, bs, d), np.uint8), np.zeros((1, hkv), np.float32)
    dk, dv, dks, dvs = up(kc), up(kc), up(ks), up(ks)
    pa.rope_append_fp8(torch.zeros(bs, 1, d, device="cuda"), up(x), up(x), dk, dv, dks, dvs, None, up(tables), up(lens), up(off))
    pa.check_error()
    _, codes, want = expected_append(x.astype(np.float64), True, kc, ks, tables, lens, off, bs)
    for c, s in ((dk, dks), (dv, dvs)):
        assert np.array_equal(s.cpu().numpy(), want)
        assert np.array_equal(c.cpu().numpy() & 0x7F, codes & 0x7F)
        assert np.array_equal(c.cpu().numpy()[codes & 0x7F != 0], codes[codes & 0x7F != 0])


def test_rope_append_fp8_special_values():
    """Zeros, infinities, NaN and values next to float32's ends; no rotation."""
    hkv, d, bs = 2, 64, 16
    x = np.zeros((6, hkv, d), np.float32)
    x[1, 0, :5] = [np.inf, -np.inf, np.nan, 2.0, -1e-30]
    x[2, 0, 0] = -8.0
    x[4, 1, :2] = [3e38, 1e-44]
    tables = np.array([[1, 2], [0, -1]], np.int32)
    lens, off = np.array([18, 4], np.int32), np.array([0, 3, 6], np.int32)
    kc, ks = np.full((3, hkv, bs, d), 0x40, np.uint8), np.full((3, hkv), 0.5, np.float32)
    dk, dv, dks, dvs = up(kc), up(kc), up(ks), up(ks)
    q = torch.zeros(6, 2, d, device="cuda")
    pa.rope_append_fp8(q, up(x), up(x), dk, dv, dks, dvs, None, up(tables), up(lens), up(off))
    pa.check_error()
    _, codes, scale = expected_append(x.astype(np.float64), True, kc, ks, tables, lens, off, bs)
    for c, s in ((dk, dks), (dv, dvs)):
        got = c.cpu().numpy()
        nan = (codes & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], codes[~nan])
        assert np.array_equal(s.cpu().numpy(), scale)


def test_rope_append_fp8_bad_tables_and_lengths():
    hkv, d, bs = 1, 64, 16
    x = torch.ones(4, hkv, d, device="cuda")
    off = up(np.array([0, 2, 4], np.int32))

    def make():
        codes = [torch.zeros(2, hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        return codes + [torch.ones(2, hkv, device="cuda") for _ in range(2)]

    def call(pool, tables, lens):
        k, v, ks, vs = pool
        pa.rope_append_fp8(x, x, x, k, v, ks, vs, None, up(np.array(tables, np.int32)), up(np.array(lens, np.int32)), off)

    pool = make()
    assert status(lambda: call(pool, [[2], [1]], [2, 2])) == 5
    assert int(pool[0][0].count_nonzero()) == 0 and int(pool[0][1].count_nonzero()) == 2 * d
    for bad in (1, 17, -5):  # below its rows, past its table, negative
        pool = make()
        assert status(lambda: call(pool, [[0], [1]], [bad, 2])) == 7
        assert int(pool[0][0].count_nonzero()) == 0 and int(pool[0][1].count_nonzero()) == 2 * d


# ---- attention -----------------------------------------------------------------------------

ATTEND = [
    # hq, hkv, old lengths, new lengths
    (1, 1, [0], [1]),
    (4, 4, [0, 126, 127, 128, 129, 255], [1, 1, 1, 1, 1, 1]),
    (28, 4, [0, 17, 300, 0, 1000, 5], [9, 0, 37, 0, 4, 128]),
    (8, 1, [2000, 3, 511], [64, 130, 1]),
    (6, 2, [0], [700]),
    (16, 8, [40] * 60, [2] * 60),
    (64, 1, [100, 9000], [5, 3]),
]


@pytest.mark.parametrize("case", ATTEND)
@pytest.mark.parametrize("dtype,d,bs,records", [("bf16", 128, 16, False), ("f16", 64, 32, True), ("f16", 128, 32, False),
                                                ("bf16", 64, 16, True)])
def test_attend_fp8(case, dtype, d, bs, records):
    hq, hkv, old, new = case
    rng = np.random.default_rng(hq * 7 + d + bs + len(old))
    lens = np.array(old) + new
    kc, vc, ks, vs, tables, lens = ref.paged(rng, lens, hkv, d, bs)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t, pad = int(off[-1]), 5
    q = torch.from_numpy(rng.standard_normal((t + pad, hq, d)).astype(np.float32)).to(T[dtype]).cuda()
    dk, dv = cache_pair(kc, vc, records)
    out = torch.full_like(q, 7.0)
    scale = d ** -0.5
    pa.attend_fp8(q, dk, dv, up(ks), up(vs), up(tables), up(lens), up(off), out=out)
    pa.check_error()
    want, bound = ref.attend(f64(q), kc, vc, ks, vs, tables, lens, off, scale, T[dtype])
    err = np.abs(f64(out)[:t] - want[:t])
    assert (err <= bound[:t]).all(), ((err - bound[:t]).max(), np.unravel_index((err - bound[:t]).argmax(), err.shape))
    assert (out[t:] == 7.0).all()


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
@pytest.mark.parametrize("dtype,q_mult,sizes", [("bf16", 3e4, (1e-6, 1e-4)), ("f16", 1.0, (1e-3, 3.0)), ("bf16", 1e-6, (2.0, 90.0))])
def test_attend_fp8_scales_far_apart(scale, dtype, q_mult, sizes):
    rng = np.random.default_rng(11)
    hq, hkv, d, bs, old, new = 4, 2, 128, 16, [200, 0, 77], [3, 150, 60]
    kc, vc, ks, vs, tables, lens = ref.paged(rng, np.array(old) + new, hkv, d, bs, sizes=sizes)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy((rng.standard_normal((off[-1], hq, d)) * q_mult).astype(np.float32)).to(T[dtype]).cuda()
    got = pa.attend_fp8(q, up(kc), up(vc), up(ks), up(vs), up(tables), up(lens), up(off), scale=scale)
    pa.check_error()
    want, bound = ref.attend(f64(q), kc, vc, ks, vs, tables, lens, off, scale, T[dtype])
    if dtype == "f16":  # outputs past f16's range are infinite
        want[np.abs(want) >= 65520] = np.copysign(np.inf, want[np.abs(want) >= 65520])
    got = f64(got)
    same = got == want
    with np.errstate(invalid="ignore"):
        assert (same | (np.abs(got - want) <= bound)).all()


def test_attend_fp8_ignores_nan_and_infinity_behind_a_row():
    """A row's result does not depend on what later rows of its request hold."""
    rng = np.random.default_rng(3)
    hq, hkv, d, bs, n, L = 4, 2, 128, 16, 20, 150
    kc, vc, ks, vs, tables, lens = ref.paged(rng, [L], hkv, d, bs)
    off = np.array([0, n], np.int32)
    for p, code in ((L - 1, 0x7F), (L - 7, 0xFF)):
        kc[tables[0, p // bs], :, p % bs, ::3] = code
        vc[tables[0, p // bs], :, p % bs, ::3] = code
    q = torch.from_numpy(rng.standard_normal((n, hq, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    q[4, 1] = float("nan")
    q[5, 2, 0] = float("inf")
    got = f64(pa.attend_fp8(q, up(kc), up(vc), up(ks), up(vs), up(tables), up(lens), up(off)))
    pa.check_error()
    with np.errstate(invalid="ignore"):
        want, bound = ref.attend(f64(q), kc, vc, ks, vs, tables, lens, off, d ** -0.5, torch.bfloat16)
        fine = np.isfinite(want)
        assert (np.abs(got - want)[fine] <= bound[fine]).all()
    assert np.isnan(got[n - 6:]).all() and np.isnan(got[4, 1]).all() and np.isnan(got[5, 2]).all()
    assert np.isfinite(got[:n - 7][[i for i in range(n - 7) if i not in (4, 5)]]).all()


def test_attend_fp8_nan_values_reach_only_their_elements():
    rng = np.random.default_rng(4)
    hkv, d, bs, n, L = 1, 64, 16, 40, 300
    kc, vc, ks, vs, tables, lens = ref.paged(rng, [L], hkv, d, bs)
    spots = [(L - 10, 3), (L - 25, 60), (100, 17)]
    for p, e in spots:
        vc[tables[0, p // bs], 0, p % bs, e] = 0x7F
    q = torch.from_numpy(rng.standard_normal((n, 2, d)).astype(np.float32)).half().cuda()
    got = f64(pa.attend_fp8(q, up(kc), up(vc), up(ks), up(vs), up(tables), up(lens), up(np.array([0, n], np.int32))))
    pa.check_error()
    want = np.zeros(got.shape, bool)
    for p, e in spots:
        for t in range(n):
            want[t, :, e] |= L - n + t >= p
    assert np.array_equal(np.isnan(got), want)


def test_attend_fp8_rows_before_position_zero_and_bad_ids():
    rng = np.random.default_rng(6)
    kc, vc, ks, vs, tables, lens = ref.paged(rng, [3, 40, 20], 2, 64, 16, nan_tail=False)
    off = np.array([0, 5, 45, 47], np.int32)  # request 0: five rows on three positions
    q = torch.randn(47, 4, 64, device="cuda").half()
    got = f64(pa.attend_fp8(q, up(kc), up(vc), up(ks), up(vs), up(tables), up(lens), up(off)))
    pa.check_error()
    want, bound = ref.attend(f64(q), kc, vc, ks, vs, tables, lens, off, 0.125, torch.float16)
    assert (got[:2] == 0).all() and (np.abs(got - want) <= bound).all()
    bad = tables.copy()
    bad[1, 1] = len(kc)
    res = []
    assert status(lambda: res.append(pa.attend_fp8(q, up(kc), up(vc), up(ks), up(vs), up(bad), up(lens), up(off)))) == 5
    keep = np.r_[0:21, 45:47]  # rows that need no position of the bad block
    assert (np.abs(f64(res[0]) - want)[keep] <= bound[keep]).all() and np.isfinite(f64(res[0])).all()
    long = lens.copy()
    long[2] = tables.shape[1] * 16 + 1
    full = np.abs(tables)  # every entry a block of the pool
    assert status(lambda: pa.attend_fp8(q, up(kc), up(vc), up(ks), up(vs), up(full), up(long), up(off))) == 7


# ---- the step ------------------------------------------------------------------------------

class Step:
    """A few requests over one pool, stepped by the operators together."""

    def __init__(self, seed, b=5, hq=8, hkv=2, d=128, bs=16, width=12, dtype=torch.bfloat16, rows=200):
        self.rng, self.b, self.hq, self.hkv, self.d, self.bs, self.rows = np.random.default_rng(seed), b, hq, hkv, d, bs, rows
        nb = b * width
        i32 = {"dtype": torch.int32, "device": "cuda"}
        self.tables, self.lens = torch.full((b, width), -1, **i32), torch.zeros(b, **i32)
        self.stack, self.free = up(self.rng.permutation(nb).astype(np.int32)), torch.full((1,), nb, **i32)
        self.new = torch.zeros(b, **i32)
        self.kc, self.vc = (torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros(nb, hkv, device="cuda") for _ in range(2))
        self.inv = pa.rope_frequencies(d, device="cuda")
        self.qkv = torch.zeros(rows, (hq + 2 * hkv) * d, dtype=dtype, device="cuda")
        self.q, self.k, self.v = (y.unflatten(1, (-1, d)) for y in self.qkv.split([hq * d, hkv * d, hkv * d], 1))
        self.out = torch.zeros(rows, hq, d, dtype=dtype, device="cuda")
        self.turned = torch.zeros_like(self.out)
        self.buffers = (self.lens, self.free, torch.empty(b + 1, **i32), torch.empty(rows, **i32),
                        torch.empty(rows, dtype=torch.int64, device="cuda"))
        self.ws = torch.empty(max(256, pa.attend_fp8_workspace_size(rows, b, hq, hkv, d, bs, width, dtype)), dtype=torch.uint8,
                              device="cuda")

    def inputs(self, new):
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.qkv.copy_(torch.from_numpy(self.rng.standard_normal(self.qkv.shape).astype(np.float32)))

    def run(self, stream=None):
        s = pa.advance_tables(self.tables, self.lens, self.new, self.stack, self.free, self.bs, self.rows, out=self.buffers,
                              stream=stream)
        pa.rope_append_fp8(self.q, self.k, self.v, self.kc, self.vc, self.ks, self.vs, self.inv, self.tables, s.context_lens,
                           s.q_offsets, query_out=self.turned, stream=stream)
        pa.attend_fp8(self.turned, self.kc, self.vc, self.ks, self.vs, self.tables, s.context_lens, s.q_offsets, out=self.out,
                      workspace=self.ws, stream=stream)
        return s

    def check(self):
        pa.check_error()
        lens, off = self.lens.cpu().numpy(), self.buffers[2].cpu().numpy()
        want, bound = ref.attend(f64(self.turned), self.kc.cpu().numpy(), self.vc.cpu().numpy(), self.ks.cpu().numpy(),
                                 self.vs.cpu().numpy(), self.tables.cpu().numpy(), lens, off, self.d ** -0.5, self.out.dtype)
        t = off[-1]
        assert (np.abs(f64(self.out)[:t] - want[:t]) <= bound[:t]).all()


STEPS = [[40, 3, 0, 17, 1], [1, 1, 1, 1, 1], [1, -1, 90, 1, 4], [1, 20, 1, -1, 1], [-1, -1, -1, -1, -1], [7, 0, 0, 0, 33]]


def test_a_step_of_the_operators_together():
    s = Step(1)
    held = np.zeros(5, int)
    for new in STEPS:
        s.inputs(new)
        s.run()
        s.check()
        held = np.where(np.array(new) < 0, 0, held + new)
        assert s.lens.cpu().tolist() == held.tolist()
    used = sum((n + 15) // 16 for n in held)
    assert int(s.free) == 60 - used


def test_a_step_over_a_16_bit_cache():
    """The tables' slots and positions feed the rotary write; decode_multi reads what it wrote."""
    s = Step(7)
    kc, vc = (torch.zeros(60, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for new in ([16, 16, 16, 16, 16], [4, 4, 4, 4, 4]):
        s.inputs(new)
        t = pa.advance_tables(s.tables, s.lens, s.new, s.stack, s.free, 16, s.rows, out=s.buffers)
        q = pa.rope_write_kv(s.q, s.k, s.v, kc, vc, s.inv, t.positions, t.slot_mapping)
    got = pa.decode_multi(q[:20].view(5, 4, 8, 128), kc, vc, s.tables, t.context_lens)
    pa.check_error()
    k, v, tab = f64(kc), f64(vc), s.tables.cpu().numpy()
    for b in range(5):
        rows = [tab[b, p // 16] for p in range(20)], [p % 16 for p in range(20)]
        for i in range(4):
            x = np.einsum("hgd,phd->hgp", f64(q)[4 * b + i].reshape(2, 4, 128), k[rows[0], :, rows[1]][:17 + i]) * 128 ** -0.5
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            vv = v[rows[0], :, rows[1]][:17 + i]
            want = np.einsum("hgp,phd->hgd", p, vv).reshape(8, 128)
            mass = np.einsum("hgp,phd->hgd", p, np.abs(vv)).reshape(8, 128)
            # half a bf16 step of the output and of P
            assert (np.abs(f64(got)[b, i] - want) <= 2.0 ** -8 * (np.abs(want) + mass) * 1.01).all()


def test_captured_steps_share_a_workspace_and_match_direct_calls():
    direct, a = Step(2), Step(2)
    b = Step(3)
    b.ws = a.ws  # two captured graphs, one workspace, replayed in turn on one stream
    graphs = []
    for s in (a, b):
        s.inputs([0] * 5)
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    direct.inputs([0] * 5)
    for new in STEPS:
        for s, g in zip((a, b), graphs):
            s.inputs(new)
            g.replay()
        direct.inputs(new)
        direct.run()
        a.check()
        b.check()
        t = int(direct.buffers[2][-1])
        assert torch.equal(a.out[:t], direct.out[:t]) and torch.equal(a.tables, direct.tables)
        assert torch.equal(a.kc, direct.kc) and torch.equal(a.ks, direct.ks)


@pytest.mark.parametrize("t", [607, 608, 611])
def test_rope_write_kv_of_many_tokens_is_that_of_each(t):
    rng = np.random.default_rng(t)
    q, k, v = qkv(rng, t, 4, 2, 64, "bf16", True)
    inv, pos = pa.rope_frequencies(64, device="cuda"), up(rng.integers(0, 9999, t).astype(np.int32))
    slots = up(rng.permutation(700)[:t].astype(np.int64))
    kc, vc = (torch.zeros(44, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc1, vc1 = torch.zeros_like(kc), torch.zeros_like(vc)
    out = pa.rope_write_kv(q, k, v, kc, vc, inv, pos, slots)
    one = [pa.rope_write_kv(q[i:i + 100], k[i:i + 100], v[i:i + 100], kc1, vc1, inv, pos[i:i + 100], slots[i:i + 100])
           for i in range(0, t, 100)]
    pa.check_error()
    assert torch.equal(out, torch.cat(one)) and torch.equal(kc, kc1) and torch.equal(vc, vc1)


def test_blocks_past_four_gigabytes():
    """The same requests in the first and in the last blocks of a pool whose K alone is larger than 2^32 bytes."""
    hq, hkv, d, bs, blocks = 8, 8, 128, 32, 140_000
    rng = np.random.default_rng(5)
    old, new = [0, 100], [70, 3]
    off, lens = up(np.array([0, 70, 73], np.int32)), up(np.array([70, 103], np.int32))
    q, k, v = qkv(rng, 73, hq, hkv, d, "bf16", True)
    inv = pa.rope_frequencies(d, device="cuda")
    low = np.array([[1, 5, 2, -1], [0, 4, 3, 6]], np.int32)
    seed = torch.randint(0, 0x78, (8, hkv, bs, d), dtype=torch.uint8, device="cuda")
    results = []
    for count, tables in ((8, low), (blocks, np.where(low >= 0, low + blocks - 8, -1).astype(np.int32))):
        kc, vc = (torch.empty(count, hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2))
        kc[-8:] = seed
        vc[-8:] = seed.flip(0)
        ks, vs = (torch.full((count, hkv), x, device="cuda") for x in (0.25, 0.5))
        turned = pa.rope_append_fp8(q, k, v, kc, vc, ks, vs, inv, up(tables), lens, off)
        out = pa.attend_fp8(turned, kc, vc, ks, vs, up(tables), lens, off)
        pos = up(np.concatenate([np.arange(a, a + n) for a, n in zip(old, new)]).astype(np.int32))
        slots = torch.arange(73, device="cuda") + (count * bs - 73)
        results.append((turned, out, kc[-8:].clone(), vc[-8:].clone(), ks[-8:].clone(), vs[-8:].clone()))
        k16, v16 = (torch.zeros(count, 2, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pa.rope_write_kv(q, k[:, :2], v[:, :2], k16, v16, inv, pos, slots)
        results[-1] += (k16[-3:].clone(), v16[-3:].clone())
        del kc, vc, k16, v16
    pa.check_error()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    steps, streams = [Step(4), Step(5)], [torch.cuda.Stream(), torch.cuda.Stream()]
    for new in STEPS:
        for s in steps:
            s.inputs(new)
        torch.cuda.synchronize()
        for s, st in zip(steps, streams):
            s.run(stream=st)
        torch.cuda.synchronize()
        for s in steps:
            s.check()


def test_attend_repeats_bit_for_bit_and_allocates_its_own_workspace():
    rng = np.random.default_rng(9)
    kc, vc, ks, vs, tables, lens = ref.paged(rng, [5000, 300, 77, 0], 2, 128, 16)
    off = up(np.array([0, 4, 100, 101, 101], np.int32))
    q = torch.randn(101, 8, 128, device="cuda").bfloat16()
    args = (q, up(kc), up(vc), up(ks), up(vs), up(tables), up(lens), off)
    first = pa.attend_fp8(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(pa.attend_fp8(*args), first)
        again = pa.attend_fp8(*args, stream=side)
        side.synchronize()
        assert torch.equal(again, first)
    pa.check_error()
