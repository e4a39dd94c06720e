"""GPU parity of the operators of a speculative step with a drafted tree against plain forms (tree_reference.py).

tree_masks, accept_tree, compact_tree: equal.  norm_rope_write_kv and attend_tree: within the bounds that
tree_reference.py derives.  All of them as a step: drafted, attended, accepted, compacted, against a host model of it;
captured and replayed; on two streams at once.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
import tree_reference as ref

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


# ---- masks -----------------------------------------------------------------------------------

@pytest.mark.parametrize("sizes,words,pad", [
    ([16] * 64, 1, 0), ([1], 1, 0), ([0, 5, 0], 1, 3), ([64, 65, 63, 1], 2, 1), ([200, 0, 129, 128, 127], 4, 700),
    ([1024, 1000, 1024, 3, 1024], 16, 5), ([0, 0], 3, 4), ([3] * 8192, 1, 2), ([], 2, 6)])
def test_tree_masks(sizes, words, pad):
    rng = np.random.default_rng(len(sizes) + words)
    off, parents = ref.trees(rng, sizes)
    lens = (rng.integers(0, 5000, len(sizes)) + sizes).astype(np.int32)
    rows = int(off[-1]) + pad
    parents = np.concatenate([parents, np.full(pad, 12345, np.int32)])  # rows behind the nodes are not read
    got = pa.tree_masks(up(parents), up(lens), up(off), words)
    pa.check_error()
    pos, seen = ref.masks(off, parents, lens, words, rows)
    assert np.array_equal(got.positions.cpu().numpy(), pos)
    assert np.array_equal(got.tree_mask.cpu().numpy(), ref.words_of(seen))


def test_tree_masks_reports_what_is_no_tree():
    off, lens = up(np.array([0, 3, 6], np.int32)), up(np.array([3, 13], np.int32))
    good = np.array([-1, 0, 1, -1, 0, 0], np.int32)
    for i, p in ((1, 1), (2, 5), (4, -2), (5, 3)):
        bad = good.copy()
        bad[i] = p
        out = []
        assert status(lambda: out.append(pa.tree_masks(up(bad), lens, off, 1))) == 7
        first = (i // 3) * 3
        want = [1, 3, 7, 1, 3, 5]
        want[i] = 1 << (i - first)  # a root
        if i == 1:
            want[2] = 6
        assert out[0].tree_mask[:, 0].tolist() == want
    # more nodes than the words hold, a length below the nodes, offsets that are no run: the other request is served
    for sizes, n, L in (([70, 6], 1, [70, 13]), ([3, 3], 1, [2, 13])):
        o, p = ref.trees(np.random.default_rng(0), sizes, "chain")
        got = (torch.full((int(o[-1]),), 77, dtype=torch.int32, device="cuda"), torch.full((int(o[-1]), n), 77, dtype=torch.int64, device="cuda"))
        assert status(lambda: pa.tree_masks(up(p), up(np.array(L, np.int32)), up(o), n, out=got)) == 7
        assert got[0][-3:].tolist() == [10, 11, 12]
    got = (torch.full((6,), 77, dtype=torch.int32, device="cuda"), torch.full((6, 1), 77, dtype=torch.int64, device="cuda"))
    for o in ([5, 3, 6], [0, 7, 6], [-1, 3, 6], [0, 3, 7]):
        assert status(lambda: pa.tree_masks(up(good), lens, up(np.array(o, np.int32)), 1, out=got)) == 7


# ---- norms with the rotary write -------------------------------------------------------------

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


@pytest.mark.parametrize("dtype,weights", [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", None)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("t,hq,hkv,d,rot,bs,fused", [
    (1, 1, 1, 64, 64, 16, False), (5, 28, 4, 128, 128, 16, True), (67, 4, 2, 64, 16, 32, True), (33, 3, 1, 80, 20, 5, False),
    (9, 2, 2, 6, 2, 1, True), (4097, 2, 1, 128, 96, 16, True), (3, 1, 1, 512, 510, 16, False), (7, 5, 3, 256, 256, 32, True),
    (12, 2, 1, 512, 128, 16, True), (40, 3, 2, 96, 0, 16, False), (611, 1, 1, 2, 2, 16, False), (0, 2, 1, 64, 64, 16, False)])
def test_norm_rope_write_kv(dtype, weights, layout, t, hq, hkv, d, rot, bs, fused):
    rng = np.random.default_rng(t + d + rot)
    q, k, v = qkv(rng, t, hq, hkv, d, dtype, fused, mult=3.0)
    nb = (t + bs - 1) // bs + 2
    pos = rng.integers(-1000, 1 << 20, t).astype(np.int32)
    pos[:1] = 2 ** 31 - 1
    slots = rng.permutation(nb * bs)[:t].astype(np.int64)
    slots[rng.random(t) < 0.2] = -1
    inv = pa.rope_frequencies(rot, device="cuda") if rot else None
    kc = torch.full((nb, hkv, bs, d), 3.0, dtype=T[dtype], device="cuda")
    vc = torch.full_like(kc, 5.0)
    qw, kw = (None, None) if weights is None else tuple(up(rng.standard_normal(d).astype(np.float32)).to(T[weights]) for _ in range(2))
    offset = 0.0 if weights is None else 0.5
    out = pa.norm_rope_write_kv(q, k, v, kc, vc, qw, kw, inv, up(pos), up(slots), eps=0.01, weight_offset=offset, layout=layout, factor=1.25)
    pa.check_error()
    # (both float64 angles are off by p * 2^-53 * inv_freq, 2e-7 each at 2^31: norm_rotate doubles the rotation's slack)
    freq = None if inv is None else inv.cpu().numpy()
    (q_want, q_slack), (k_want, k_slack) = (
        ref.norm_rotate(f64(x), None if w is None else f64(w), 0.01, offset, pos, freq, layout, 1.25) for x, w in ((q, qw), (k, kw)))
    near(f64(out), q_want, q_slack, dtype)
    kw_, vw, sl = np.full(kc.shape, 3.0), np.full(kc.shape, 5.0), np.zeros(kc.shape)
    use = slots >= 0
    kw_[slots[use] // bs, :, slots[use] % bs] = k_want[use]
    sl[slots[use] // bs, :, slots[use] % bs] = k_slack[use]
    vw[slots[use] // bs, :, slots[use] % bs] = f64(v)[use]
    near(f64(kc), kw_, sl, dtype)
    assert np.array_equal(f64(vc), vw)


def test_norm_rope_write_kv_without_a_norm_to_speak_of_is_the_rotary_write():
    """Heads whose elements are +-1 have norm 1: with weights of one and no eps, the float32 results are rope_write_kv's."""
    rng = np.random.default_rng(1)
    q, k, v = (up(rng.choice([-1.0, 1.0], (50, h, 64)).astype(np.float32)) for h in (6, 2, 2))
    inv, pos, slots = pa.rope_frequencies(64, device="cuda"), up(rng.integers(0, 9999, 50).astype(np.int32)), up(rng.permutation(64)[:50].astype(np.int64))
    caches = [torch.zeros(4, 2, 16, 64, device="cuda") for _ in range(4)]
    one = pa.rope_write_kv(q, k, v, caches[0], caches[1], inv, pos, slots)
    two = pa.norm_rope_write_kv(q, k, v, caches[2], caches[3], None, None, inv, pos, slots, eps=0.0)
    pa.check_error()
    assert torch.equal(one, two) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_norm_rope_write_kv_in_place_bad_slot_and_rows_of_zeros_infinities_and_nan():
    rng = np.random.default_rng(2)
    q, k, v = qkv(rng, 7, 4, 2, 64, "bf16", False)
    q[0] = 0
    k[1, 0, 5] = float("inf")
    k[2, 1, 6] = float("nan")
    kc, vc = (torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.ones(64, device="cuda")
    inv, pos = pa.rope_frequencies(64, device="cuda"), up(np.arange(7, dtype=np.int32))
    slots = np.arange(7, dtype=np.int64)
    want = pa.norm_rope_write_kv(q, k, v, kc, vc, w, None, inv, pos, up(slots))
    assert (want[0] == 0).all() and torch.isnan(kc[0, 0, 1]).any() and torch.isnan(kc[0, 1, 2]).all()
    assert torch.isfinite(kc[0, 1, 1]).all() and torch.isfinite(kc[0, 0, 2]).all() and torch.isfinite(kc[0, :, 3:7]).all()
    kept = kc.clone()
    slots[3] = 32
    same = q.clone()
    assert status(lambda: pa.norm_rope_write_kv(same, k, v, kc, vc, w, None, inv, pos, up(slots), query_out=same)) == 6
    assert torch.equal(same, want) and torch.equal(kc.nan_to_num(), kept.nan_to_num())


def test_norm_rope_write_kv_of_views_at_odd_addresses():
    rng = np.random.default_rng(6)
    t, hq, hkv, d = 21, 3, 2, 64
    base = torch.from_numpy(rng.standard_normal((t, (hq + 2 * hkv) * d + 5)).astype(np.float32)).half().cuda()
    q, k, v = (y.unflatten(1, (-1, d)) for y in base[:, 3:3 + (hq + 2 * hkv) * d].split([hq * d, hkv * d, hkv * d], 1))
    w = torch.randn(2 * d + 1, device="cuda").half()
    inv, pos, slots = pa.rope_frequencies(d, device="cuda"), up(np.arange(t, dtype=np.int32)), up(np.arange(t, dtype=np.int64))
    caches = [torch.zeros(2, hkv, 16, d, dtype=torch.float16, device="cuda") for _ in range(4)]
    odd = pa.norm_rope_write_kv(q, k, v, caches[0], caches[1], w[1:d + 1], w[d + 1:], inv, pos, slots)
    even = pa.norm_rope_write_kv(q.contiguous(), k.contiguous(), v.contiguous(), caches[2], caches[3], w[1:d + 1].clone(),
                                 w[d + 1:].clone(), inv, pos, slots)
    pa.check_error()
    want, slack = ref.norm_rotate(f64(q), f64(w[1:d + 1]), 1e-6, 0.0, np.arange(t), inv.cpu().numpy(), "half", 1.0)
    near(f64(odd), want, slack, "f16")
    near(f64(even), want, slack, "f16")
    assert torch.equal(caches[1], caches[3])


# ---- attention ---------------------------------------------------------------------------------

def attend_case(rng, hq, hkv, d, bs, dtype, old, new, kind="mixed", pad=3, **more):
    """Inputs of a call on the GPU, and the wanted (out, bound)."""
    lens = np.array(old) + new
    kc, vc, tables, lens = ref.paged(rng, lens, hkv, d, bs, T[dtype], **more)
    off, parents = ref.trees(rng, new, kind)
    t, words = int(off[-1]) + pad, max(1, (max(new) + 63) // 64)
    _, seen = ref.masks(off, parents, lens, words, t)
    q = torch.from_numpy(rng.standard_normal((t, hq, d)).astype(np.float32)).to(T[dtype])
    return {"q": q, "kc": kc, "vc": vc, "tables": tables, "lens": lens, "off": off, "seen": seen, "new": new}


def attend(c, **more):
    out = torch.full(tuple(c["q"].shape), 9.0, dtype=c["q"].dtype, device="cuda")
    pa.attend_tree(c["q"].cuda(), c["kc"].cuda(), c["vc"].cuda(), up(ref.words_of(c["seen"])), up(c["tables"]), up(c["lens"]), up(c["off"]),
                   out=out, **more)
    return out


def check(c, out, scale=None, rows=None):
    d = c["q"].shape[2]
    want, bound = ref.attend(f64(c["q"]), f64(c["kc"]), f64(c["vc"]), c["tables"], c["lens"], c["off"], c["seen"],
                             d ** -0.5 if scale is None else scale, c["q"].dtype)
    t = int(c["off"][-1])
    got = f64(out)
    assert (got[t:] == 9.0).all()
    rows = slice(0, t) if rows is None else rows
    assert np.isfinite(got[rows]).all()
    err = np.abs(got[rows] - want[rows])
    assert (err <= bound[rows]).all(), (err / np.maximum(bound[rows], 1e-30)).max()


ATTEND = [
    # hq, hkv, d, bs, cached, nodes
    (4, 2, 128, 16, [0, 5, 16, 31], [1, 1, 1, 1]),
    (7, 1, 128, 16, [0, 15, 40, 0, 3], [33, 0, 100, 0, 13]),
    (8, 8, 64, 32, [0, 33, 1], [32, 31, 200]),
    (6, 2, 64, 16, [900], [1]),
    (28, 4, 128, 16, [700, 1000, 128, 127, 129], [16, 16, 16, 16, 16]),
    (28, 4, 128, 32, [1500, 60], [64, 128]),
    (8, 1, 128, 16, [300, 0, 20], [70, 129, 2]),
    (16, 4, 64, 32, [0, 100, 500, 0, 7, 31, 32, 33], [40, 0, 1, 3, 17, 1, 32, 0]),
    (4, 4, 128, 16, [5000, 100], [3, 1]),
    (2, 1, 64, 16, [10] * 300, [1, 0, 3, 2, 5, 7] * 50),
    (2, 2, 128, 32, [40], [1024]),
    (64, 1, 128, 16, [200, 0], [9, 5]),
    (2, 1, 64, 16, [60000], [3]),  # one unit in the shares of more than 32 SMs
    (3, 1, 64, 32, [5, 130, 0] * 600, [1, 0, 2] * 600),  # several requests to a thread that adds up costs
    (300, 1, 128, 16, [40, 700], [2, 1]),  # more heads to a node than rows to a tile
]


@pytest.mark.parametrize("case", ATTEND)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_tree(case, dtype):
    hq, hkv, d, bs, old, new = case
    rng = np.random.default_rng(len(old) * 100 + d + bs)
    c = attend_case(rng, hq, hkv, d, bs, dtype, old, new)
    out = attend(c)
    pa.check_error()
    check(c, out)


@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32)])
@pytest.mark.parametrize("old", [0, 3, 128, 250])
def test_attend_tree_takes_any_mask_and_rows_that_see_nothing(d, bs, old):
    """Random bits, nodes after the row among them, bits behind the last node, empty rows (zeros where nothing is cached)."""
    rng = np.random.default_rng(old + d)
    c = attend_case(rng, 6, 2, d, bs, "bf16", [old, old + 1, 0], [70, 5, 131])
    c["seen"] = rng.random(c["seen"].shape) < 0.3
    c["seen"][::3] = False
    c["seen"][5] = True
    out = attend(c)
    pa.check_error()
    check(c, out)
    if old == 0:
        assert (out[3] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("old", [0, 10, 120, 1000])
def test_nodes_that_a_row_does_not_see_do_not_reach_it(dtype, old):
    """NaN and infinities in K and V of some nodes: rows that do not see them are as if they were not there; rows that do get
    what the sums give."""
    rng = np.random.default_rng(old)
    hq, hkv, d, bs = 14, 2, 128, 16
    c = attend_case(rng, hq, hkv, d, bs, dtype, [old, 40], [20, 80], kind="random")
    off, lens, tables = c["off"], c["lens"], c["tables"]

    def place(b, node):
        p = int(lens[b]) - int(off[b + 1] - off[b]) + node
        return int(tables[b, p // bs]), p % bs

    inf, nan = float("inf"), float("nan")
    hurt = {(0, 4): ("v", 3, nan), (0, 9): ("k", 0, nan), (0, 12): ("v", 100, inf), (1, 7): ("v", 64, -inf), (1, 50): ("k", 9, inf),
            (1, 79): ("v", 127, nan), (1, 33): ("v", 0, inf), (1, 34): ("v", 0, -inf)}
    for (b, node), (which, e, x) in hurt.items():
        blk, o = place(b, node)
        c["kc" if which == "k" else "vc"][blk, :, o, e] = x
    out = f64(attend(c))
    pa.check_error()
    sees = np.zeros((int(off[-1]), len(hurt)), bool)
    for i, (b, node) in enumerate(hurt):
        sees[off[b]:off[b + 1], i] = c["seen"][off[b]:off[b + 1], node]
    clean = np.flatnonzero(~sees.any(1))
    assert 10 < len(clean) < len(sees)
    check(c, torch.from_numpy(out), rows=clean)
    names = list(hurt)
    for t in np.flatnonzero(sees.any(1)):
        marks = {names[i]: hurt[names[i]] for i in np.flatnonzero(sees[t])}
        if any(w == "k" for w, _, _ in marks.values()):
            assert np.isnan(out[t]).all() or any(x == inf and w == "k" for w, _, x in marks.values())
            continue
        for e in range(d):
            here = [x for _, at, x in marks.values() if at == e]
            if not here:
                assert np.isfinite(out[t, :, e]).all()
            elif any(x != x for x in here) or len(set(here)) > 1:
                assert np.isnan(out[t, :, e]).all()
            else:
                assert (out[t, :, e] == here[0]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.09, 1.0, 3.0])
def test_attend_tree_scales(dtype, scale):
    rng = np.random.default_rng(8)
    c = attend_case(rng, 8, 2, 128, 16, dtype, [300, 3], [9, 70])
    out = attend(c, scale=scale)
    pa.check_error()
    check(c, out, scale=scale)


def test_attend_tree_maxima_that_rise_along_the_context():
    """Keys that grow with their position: the reference of the exponents is replaced again and again."""
    rng = np.random.default_rng(9)
    c = attend_case(rng, 4, 1, 128, 16, "bf16", [3000], [6])
    pos = np.arange(3006)
    grow = torch.from_numpy(np.linspace(0.01, 12.0, 3006)).float()
    rows = c["kc"].float()
    rows[c["tables"][0, pos // 16], 0, pos % 16] *= grow[:, None]
    c["kc"] = rows.bfloat16()
    out = attend(c)
    pa.check_error()
    check(c, out)


def test_attend_tree_reports_bad_tables_and_lengths():
    rng = np.random.default_rng(11)
    base = attend_case(rng, 4, 2, 128, 16, "bf16", [100, 300], [5, 20], fill=0.0)

    def with_(**changes):
        return {**base, **changes}

    tables = base["tables"].copy()
    tables[0, 2], tables[1, 7] = -1, len(base["kc"])
    c = with_(tables=tables)
    out = []
    assert status(lambda: out.append(attend(c))) == 5
    check(c, out[0])  # masked positions
    # a length past the table is clamped, one below the nodes starts before position 0
    c = with_(lens=np.array([3, 320 + 16], np.int32), tables=base["tables"][:, :20])
    out = []
    assert status(lambda: out.append(attend(c))) == 7
    clamped = with_(lens=np.array([3, 320], np.int32), tables=base["tables"][:, :20])
    seen = clamped["seen"].copy()
    want, bound = ref.attend(f64(c["q"]), f64(c["kc"]), f64(c["vc"]), clamped["tables"], clamped["lens"], c["off"], seen, 128 ** -0.5, torch.bfloat16)
    got = f64(out[0])
    assert (np.abs(got[5:25] - want[5:25]) <= bound[5:25]).all()
    # node j of the first request sits at position j - 2
    assert np.isfinite(got[:5]).all() and (got[0] == 0).all()
    # nodes past the words are seen by nobody
    c = attend_case(rng, 4, 2, 128, 16, "bf16", [50], [70], kind="chain", fill=0.0)
    c["seen"] = c["seen"][:, :64]
    out = []
    assert status(lambda: out.append(attend(c))) == 7
    check(c, out[0])
    # offsets that are no run: the other requests are served, and nothing else is written
    for bad in ([7, 5, 25], [0, 40, 25], [-3, 5, 25], [0, 5, 29]):
        c = with_(off=np.array(bad, np.int32))
        out = []
        assert status(lambda: out.append(attend(c))) == 7
        served = [b for b in range(2) if 0 <= bad[b] <= bad[b + 1] <= 28 and bad[b + 1] - bad[b] <= 64]
        got, touched = f64(out[0]), np.zeros(28, bool)
        for b in served:
            touched[bad[b]:bad[b + 1]] = True
        assert (got[~touched] == 9.0).all()


def test_attend_tree_refuses_a_small_workspace_and_repeats_bit_for_bit():
    rng = np.random.default_rng(12)
    c = attend_case(rng, 28, 4, 128, 16, "bf16", [5000, 300, 77, 0], [16, 40, 1, 0])
    need = pa.attend_tree_workspace_size(c["q"].shape[0], 4, 28, 4, 128, 16, c["tables"].shape[1], torch.bfloat16)
    if need > 0:
        with pytest.raises(pa.PAError) as e:
            attend(c, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == 1 and str(need) in str(e.value)
    first, side = attend(c), torch.cuda.Stream()
    dirty = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(attend(c, workspace=dirty), first)
        torch.cuda.synchronize()
        again = attend(c, stream=side)
        side.synchronize()
        assert torch.equal(again, first)
    pa.check_error()
    check(c, first)


def test_attend_tree_leaves_everything_as_it_was_without_nodes_and_with_overlapping_runs():
    rng = np.random.default_rng(14)
    c = attend_case(rng, 4, 2, 128, 16, "bf16", [100, 300], [5, 20], fill=0.0)
    c["off"] = np.zeros(3, np.int32)
    assert (attend(c) == 9.0).all()
    pa.check_error()
    c["off"], c["lens"] = np.zeros(1, np.int32), np.zeros(0, np.int32)
    c["tables"] = np.zeros((0, 3), np.int32)
    assert (attend(c) == 9.0).all()
    pa.check_error()
    # more rows in the runs than there are tokens: nothing is done
    c = attend_case(rng, 4, 2, 128, 16, "bf16", [100] * 3, [5, 5, 5], pad=0, fill=0.0)
    c["off"] = np.array([0, 14, 1, 15], np.int32)
    out = []
    assert status(lambda: out.append(attend(c))) == 7
    assert (out[0] == 9.0).all()


def test_attend_tree_of_one_node_is_a_decode_step():
    """One node that sees itself is a token of a decode step: the decode call's result, within both bounds."""
    rng = np.random.default_rng(13)
    c = attend_case(rng, 28, 4, 128, 16, "bf16", [0, 15, 700, 3000, 64], [1] * 5, pad=0)
    one = attend(c)
    two = pa.decode(c["q"].cuda(), c["kc"].cuda(), c["vc"].cuda(), up(c["tables"]), up(c["lens"]))
    pa.check_error()
    check(c, one)
    _, bound = ref.attend(f64(c["q"]), f64(c["kc"]), f64(c["vc"]), c["tables"], c["lens"], c["off"], c["seen"], 128 ** -0.5, torch.bfloat16)
    assert (np.abs(f64(one) - f64(two)) <= 2 * bound).all()


def test_blocks_past_four_gigabytes():
    """The same requests in the first and in the last blocks of a pool whose K alone is larger than 2^32 bytes."""
    hq, hkv, d, bs, blocks = 8, 8, 128, 32, 140_000
    rng = np.random.default_rng(5)
    off, parents = ref.trees(rng, [20, 3], "random")
    lens = np.array([70, 103], np.int32)
    _, seen = ref.masks(off, parents, lens, 1, 23)
    q, mask = torch.randn(23, hq, d, device="cuda").bfloat16(), up(ref.words_of(seen))
    low = np.array([[1, 5, 2, -1], [0, 4, 3, 6]], np.int32)
    seed = torch.randn(8, hkv, bs, d, device="cuda").bfloat16()
    accepted, count = up(np.array([[0, 3, 9, 19], [0, 2, -1, -1]], np.int32)), up(np.array([4, 2], np.int32))
    results = []
    for n, tables in ((8, low), (blocks, np.where(low >= 0, low + blocks - 8, -1).astype(np.int32))):
        kc, vc = (torch.empty(n, hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kc[-8:] = seed
        vc[-8:] = seed.flip(0)
        out = pa.attend_tree(q, kc, vc, mask, up(tables), up(lens), up(off))
        pos = np.concatenate([np.arange(50, 70), np.arange(100, 103)])
        slots = tables[np.repeat([0, 1], [20, 3]), pos // bs].astype(np.int64) * bs + pos % bs
        stack, free = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.norm_rope_write_kv(q, q, q, kc, vc, None, None, pa.rope_frequencies(d, device="cuda"), up(pos.astype(np.int32)), up(slots))
        state = pa.compact_tree([kc], [vc], up(slots), up(off), accepted, count, up(tables), up(lens), stack, free)
        results.append((out, kc[-8:].clone(), vc[-8:].clone(), state.context_lens, state.num_free))
        del kc, vc
    pa.check_error()
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ---- acceptance -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("sizes,depth,vocab", [
    ([16] * 64, 8, 3), ([1], 1, 5), ([0, 5, 0], 4, 2), ([200, 0, 129, 64, 65], 16, 4), ([1024, 1000, 1024, 3, 1024], 1024, 1),
    ([3] * 8192, 2, 3), ([40] * 10, 3, 1), ([], 4, 2)])
def test_accept_tree(dtype, sizes, depth, vocab):
    rng = np.random.default_rng(len(sizes) + depth)
    off, parents = ref.trees(rng, sizes)
    t = int(off[-1])
    big = 0 if dtype == torch.int32 else 1 << 40
    tokens, choices = (rng.integers(0, vocab, t) + big for _ in range(2))
    got = pa.accept_tree(up(parents), up(tokens).to(dtype), up(choices).to(dtype), up(off), depth)
    pa.check_error()
    accepted, count, token = ref.accept(off, parents, tokens, choices, depth)
    assert np.array_equal(got.accepted.cpu().numpy(), accepted) and np.array_equal(got.num_accepted.cpu().numpy(), count)
    assert got.next_tokens.dtype == dtype and np.array_equal(got.next_tokens.cpu().numpy(), token)


def test_accept_tree_reports_what_is_no_tree():
    off = up(np.array([0, 3, 6], np.int32))
    tokens, good = up(np.full(6, 7)), np.array([-1, 0, 1, -1, 0, 1], np.int32)
    for i, p, want in ((1, 1, [1, 3]), (2, 4, [2, 3]), (4, -3, [3, 1]), (3, 0, [3, 3])):
        bad = good.copy()
        bad[i] = p
        got = []
        assert status(lambda: got.append(pa.accept_tree(up(bad), tokens, tokens, off, 4))) == 7
        assert got[0].num_accepted.tolist() == want
    for o, want in (([5, 3, 6], [0, 3]), ([0, 7, 6], [0, 0]), ([0, 3, 7], [3, 0])):
        got = []
        assert status(lambda: got.append(pa.accept_tree(up(good), tokens, tokens, up(np.array(o, np.int32)), 4))) == 7
        assert got[0].num_accepted.tolist() == want and got[0].accepted[np.array(want) == 0].eq(-1).all()
    long = up(np.arange(-1, 1024, dtype=np.int32))
    got = []
    many = torch.zeros(1025, dtype=torch.int64, device="cuda")
    assert status(lambda: got.append(pa.accept_tree(long, many, many, up(np.array([0, 1025], np.int32)), 4))) == 7
    assert got[0].num_accepted.tolist() == [0] and got[0].next_tokens.tolist() == [-1]


# ---- compaction -----------------------------------------------------------------------------------

def compact_case(rng, layers, hkv, d, bs, dtype, old, new, depth):
    lens = np.array(old) + new
    _, _, tables, lens = ref.paged(rng, lens, 1, 1, bs, torch.float32)
    used = (lens + bs - 1) // bs
    nb = int(used.sum()) + 3
    keys, values = (torch.from_numpy(rng.integers(-100, 100, (layers, nb, hkv, bs, d)).astype(np.float32)).to(T[dtype]) for _ in range(2))
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.repeat(np.arange(len(new)), new)
    pos = np.array(old)[seq] + np.arange(off[-1]) - off[seq]
    slots = tables[seq, pos // bs].astype(np.int64) * bs + pos % bs
    accepted, count = np.full((len(new), depth), -1, np.int32), np.zeros(len(new), np.int32)
    for b, n in enumerate(new):
        count[b] = rng.integers(0, min(n, depth) + 1)
        accepted[b, :count[b]] = np.sort(rng.permutation(n)[:count[b]])
    held = set(tables[b, j] for b in range(len(new)) for j in range(used[b]))
    free = [i for i in range(nb) if i not in held]
    stack = np.full(nb, -9, np.int32)
    stack[:len(free)] = free
    return {"keys": keys, "values": values, "slots": slots, "off": off, "accepted": accepted, "count": count, "tables": tables, "lens": lens,
            "stack": stack, "free": len(free), "bs": bs}


def compact(c, keys, values, in_place=False, **more):
    lens, stack, free = up(c["lens"]), up(c["stack"]), torch.tensor([c["free"]], dtype=torch.int32, device="cuda")
    got = pa.compact_tree(keys, values, up(c["slots"]), up(c["off"]), up(c["accepted"]), up(c["count"]), up(c["tables"]), lens, stack, free,
                          out=(lens, free) if in_place else None, **more)
    return got, stack


COMPACT = [
    # layers, hkv, d, bs, cached, nodes, depth
    (3, 4, 128, 16, [100, 5, 16, 0], [16, 16, 16, 16], 5),
    (1, 1, 64, 16, [0], [1], 1),
    (28, 2, 80, 32, [31, 0, 64, 7, 9], [40, 0, 3, 64, 1], 16),
    (2, 3, 6, 5, [4, 9], [33, 70], 40),
    (5, 8, 128, 16, [15] * 60, [1, 0, 9, 20, 64, 5] * 10, 12),
    (1, 1, 2, 1, [3, 4], [200, 1024], 1024),
    (2, 1, 8, 16, [1] * 8192, [2] * 8192, 2),
]


@pytest.mark.parametrize("case", COMPACT)
@pytest.mark.parametrize("dtype,in_place", [("f32", True), ("bf16", False), ("f16", True)])
def test_compact_tree(case, dtype, in_place):
    rng = np.random.default_rng(case[0] + case[2])
    c = compact_case(rng, case[0], case[1], case[2], case[3], dtype, case[4], case[5], case[6])
    keys, values = c["keys"].cuda(), c["values"].cuda()
    if not in_place:
        keys, values = list(keys.unbind(0)), list(values.unbind(0))
    got, stack = compact(c, keys, values, in_place)
    pa.check_error()
    k, v = f64(c["keys"]), f64(c["values"])
    lens, want_stack, free = ref.compact([k, v], c["slots"], c["off"], c["accepted"], c["count"], c["tables"], c["lens"], c["stack"], c["free"], c["bs"])
    if not in_place:
        keys, values = torch.stack(keys), torch.stack(values)
    assert np.array_equal(f64(keys), k) and np.array_equal(f64(values), v)
    assert got.context_lens.cpu().tolist() == lens.tolist() and int(got.num_free) == free
    assert np.array_equal(stack.cpu().numpy(), want_stack)


def test_compact_tree_of_caches_at_odd_addresses():
    rng = np.random.default_rng(3)
    c = compact_case(rng, 2, 2, 8, 16, "f16", [3, 40], [30, 9], 8)
    flat = [torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda") for x in (c["keys"], c["values"])]
    views = [f[1:].view(x.shape) for f, x in zip(flat, (c["keys"], c["values"]))]
    for view, x in zip(views, (c["keys"], c["values"])):
        view.copy_(x)
    compact(c, *views)
    pa.check_error()
    k, v = f64(c["keys"]), f64(c["values"])
    ref.compact([k, v], c["slots"], c["off"], c["accepted"], c["count"], c["tables"], c["lens"], c["stack"], c["free"], c["bs"])
    assert np.array_equal(f64(views[0]), k) and np.array_equal(f64(views[1]), v)


@pytest.mark.parametrize("what,code", [("order", 7), ("twice", 7), ("past", 7), ("negative", 7), ("many", 7), ("below", 7), ("short", 7),
                                       ("wide", 7), ("run", 7), ("table", 5), ("room", 5), ("count", 5), ("slot", 6), ("unmapped", 6)])
def test_compact_tree_reports_and_keeps_what_it_cannot_do(what, code):
    rng = np.random.default_rng(4)
    c = compact_case(rng, 2, 2, 16, 16, "bf16", [20, 30], [30, 40], 4)
    c["accepted"][:], c["count"][:] = [[0, 3, 9, 20], [0, 1, 7, 39]], 4
    tables = c["tables"]
    if what == "order":
        c["accepted"][0, 2] = 2
    elif what == "twice":
        c["accepted"][0, 2] = 3
    elif what == "past":
        c["accepted"][0, 3] = 30
    elif what == "negative":
        c["accepted"][0, 0] = -1
    elif what == "many":
        c["count"][0] = 5
    elif what == "below":
        c["count"][0] = -1
    elif what == "short":
        c["lens"][0] = 29
    elif what == "wide":
        c["lens"][0] = tables.shape[1] * 16 + 1
    elif what == "run":
        c["off"][0] = 31
    elif what == "table":
        tables[0, 3] = len(c["stack"])
    elif what == "room":
        c["free"] = len(c["stack"])
    elif what == "count":
        c["free"] = -1
    elif what == "slot":
        c["slots"][3] = len(c["stack"]) * 16
    elif what == "unmapped":
        c["slots"][1] = -1
    keys, values = c["keys"].cuda(), c["values"].cuda()
    got = []
    assert status(lambda: got.append(compact(c, keys, values))) == code
    (state, stack), = got
    lens, free = state.context_lens.cpu().tolist(), int(state.num_free)
    if what in ("room", "count"):
        assert lens == c["lens"].tolist() and free == c["free"] and np.array_equal(stack.cpu().numpy(), c["stack"])
        return
    second = 30 + 4
    assert lens[1] == second
    if what in ("slot", "unmapped"):
        assert lens[0] == 24
    else:
        assert lens[0] == c["lens"][0]
        gone = tables[1, 3:5].tolist()
        assert free == c["free"] + 2 and stack[c["free"]:free].tolist() == gone
    # the second request's nodes moved, the first's only where its branch is one
    k = f64(c["keys"])
    moved = k.copy()
    for j, a in enumerate([0, 1, 7, 39]):
        s, d = c["slots"][30 + a], c["slots"][30 + j]
        moved[:, d // 16, :, d % 16] = k[:, s // 16, :, s % 16]
    blocks = tables[1, :5]
    assert np.array_equal(f64(keys)[:, blocks], moved[:, blocks])
    if what in ("order", "twice", "past", "negative", "many", "below", "run"):
        rest = [i for i in range(k.shape[1]) if i not in blocks]
        assert np.array_equal(f64(keys)[:, rest], k[:, rest])


# ---- all of them as a step ---------------------------------------------------------------------------

class Step:
    """Requests whose trees are drafted by a rule, verified by one layer of attention per cache, and compacted; the host model
    keeps, per request, the rows of K and V that its cache has to hold."""

    def __init__(self, seed, b=5, hq=8, hkv=2, d=64, bs=16, width=12, rows=96, layers=3, depth=6):
        self.rng = np.random.default_rng(seed)
        self.b, self.hq, self.hkv, self.d, self.bs, self.rows, self.layers, self.depth = b, hq, hkv, d, bs, rows, layers, depth
        i32 = {"dtype": torch.int32, "device": "cuda"}
        blocks = b * width
        self.tables, self.lens = torch.full((b, width), -1, **i32), torch.zeros(b, **i32)
        self.stack, self.free = up(self.rng.permutation(blocks).astype(np.int32)), torch.tensor([blocks], **i32)
        self.kc, self.vc = (torch.full((layers, blocks, hkv, bs, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.new, self.parents = torch.zeros(b, **i32), torch.zeros(rows, **i32)
        self.tokens, self.choices = (torch.zeros(rows, dtype=torch.int64, device="cuda") for _ in range(2))
        self.inv = pa.rope_frequencies(d, device="cuda")
        self.qw, self.kw = (torch.rand(d, device="cuda") + 0.5 for _ in range(2))
        self.qkv = torch.zeros(layers, rows, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device="cuda")
        self.buffers = (self.lens, self.free, torch.empty(b + 1, **i32), torch.empty(rows, **i32),
                        torch.empty(rows, dtype=torch.int64, device="cuda"))
        self.masks = (torch.empty(rows, **i32), torch.empty(rows, 1, dtype=torch.int64, device="cuda"))
        self.path = (torch.empty(b, depth, **i32), torch.empty(b, **i32), torch.empty(b, dtype=torch.int64, device="cuda"))
        self.turned, self.out = (torch.zeros(layers, rows, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.ws = torch.empty(max(256, pa.attend_tree_workspace_size(rows, b, hq, hkv, d, bs, width, torch.bfloat16)), dtype=torch.uint8,
                              device="cuda")
        self.held = [[] for _ in range(b)]  # (K rows, V rows) of every cached position: [layers, hkv, d] each

    def inputs(self, new):
        self.sizes = np.array(new)
        off, parents = ref.trees(self.rng, np.maximum(new, 0))
        t = int(off[-1])
        choices = self.rng.integers(0, 3, self.rows)
        tokens = self.rng.integers(0, 3, self.rows)
        for dst, src in ((self.new, np.array(new, np.int32)), (self.parents, np.concatenate([parents, np.zeros(self.rows - t, np.int32)])),
                         (self.tokens, tokens), (self.choices, choices)):
            dst.copy_(torch.from_numpy(np.ascontiguousarray(src)))
        self.qkv.copy_(torch.from_numpy(self.rng.standard_normal(self.qkv.shape).astype(np.float32)))
        self.off, self.host_parents = off, parents
        self.want_path = ref.accept(off, parents, tokens[:t], choices[:t], self.depth)

    def run(self, stream=None):
        s = pa.advance_tables(self.tables, self.lens, self.new, self.stack, self.free, self.bs, self.rows, out=self.buffers, stream=stream)
        m = pa.tree_masks(self.parents, s.context_lens, s.q_offsets, 1, out=self.masks, stream=stream)
        for l in range(self.layers):
            q, k, v = (y.unflatten(1, (-1, self.d)) for y in self.qkv[l].split([self.hq * self.d, self.hkv * self.d, self.hkv * self.d], 1))
            pa.norm_rope_write_kv(q, k, v, self.kc[l], self.vc[l], self.qw, self.kw, self.inv, m.positions, s.slot_mapping,
                                  query_out=self.turned[l], stream=stream)
            pa.attend_tree(self.turned[l], self.kc[l], self.vc[l], m.tree_mask, self.tables, s.context_lens, s.q_offsets, out=self.out[l],
                           workspace=self.ws, stream=stream)
        p = pa.accept_tree(self.parents, self.tokens, self.choices, s.q_offsets, self.depth, out=self.path, stream=stream)
        pa.compact_tree(self.kc, self.vc, s.slot_mapping, s.q_offsets, p.accepted, p.num_accepted, self.tables, s.context_lens, self.stack,
                        self.free, out=(self.lens, self.free), stream=stream)

    def check(self):
        pa.check_error()
        accepted, count, token = self.want_path
        assert np.array_equal(self.path[0].cpu().numpy(), accepted) and np.array_equal(self.path[1].cpu().numpy(), count)
        assert np.array_equal(self.path[2].cpu().numpy(), token)
        cached = np.array([len(h) for h in self.held])
        gone = self.sizes < 0
        nodes = np.maximum(self.sizes, 0)
        pos, seen = ref.masks(self.off, self.host_parents, np.where(gone, 0, cached + nodes), 1, self.rows)
        assert np.array_equal(self.masks[0].cpu().numpy(), pos)
        # K and V of the step's nodes from the definition, what is cached from the model
        heads = self.qkv.double().cpu().numpy().reshape(self.layers, self.rows, -1, self.d)
        lens = []
        for b in range(self.b):
            if gone[b]:
                self.held[b] = []
            lens.append(len(self.held[b]) + count[b])
        t = int(self.off[-1])
        kc, vc, tables = f64(self.kc), f64(self.vc), self.tables.cpu().numpy()
        got, rounded = f64(self.out), f64(self.turned)
        new_k = np.zeros((self.layers, t, self.hkv, self.d))
        new_v = heads[:, :t, self.hq + self.hkv:]
        for l in range(self.layers):
            for part, weight, to in ((slice(0, self.hq), self.qw, rounded[l][:t]), (slice(self.hq, self.hq + self.hkv), self.kw, None)):
                want, slack = ref.norm_rotate(heads[l, :t, part], f64(weight), 1e-6, 0.0, pos[:t], self.inv.cpu().numpy(), "half", 1.0)
                if to is not None:
                    near(to, want, slack, "bf16")
                else:
                    new_k[l] = want
        for b in range(self.b):
            lo, n = int(self.off[b]), int(nodes[b])
            # attention: cached rows and the nodes' own, as a cache of one block table
            L = len(self.held[b]) + n
            if n:
                k = np.stack([h[0] for h in self.held[b]] + list(new_k[:, lo:lo + n].swapaxes(0, 1)))  # [L, layers, hkv, d]
                v = np.stack([h[1] for h in self.held[b]] + list(new_v[:, lo:lo + n].swapaxes(0, 1)))
                for l in range(self.layers):
                    want, bound = ref.attend(rounded[l][lo:lo + n], k[:, l][:, :, None], v[:, l][:, :, None], np.arange(L)[None], np.array([L]),
                                             np.array([0, n]), seen[lo:lo + n], self.d ** -0.5, torch.bfloat16)
                    # new_k is not rounded to bf16 here: half a step of it moves a score by 2^-9 sum |q k| and more
                    s = self.d ** -0.5 * np.einsum("thd,phd->tph", np.abs(rounded[l][lo:lo + n]), np.repeat(np.abs(k[:, l]), self.hq // self.hkv, 1)).max((1, 2))
                    mass = np.abs(v[:, l]).max()
                    assert (np.abs(got[l][lo:lo + n] - want) <= bound + 2 * 2.0 ** -8 * (s * mass)[:, None, None]).all()
            for j in range(count[b]):
                node = lo + accepted[b, j]
                self.held[b].append((new_k[:, node], new_v[:, node]))
            assert len(self.held[b]) == lens[b]
            for p, (k, v) in enumerate(self.held[b]):
                blk, o = tables[b, p // self.bs], p % self.bs
                near(kc[:, blk, :, o], k, 1e-5 * np.abs(k).max(), "bf16")
                assert np.array_equal(vc[:, blk, :, o], v)
                self.held[b][p] = (kc[:, blk, :, o].copy(), v)  # as stored: later steps see the rounded keys
        assert self.lens.cpu().tolist() == lens
        used = [set(tables[b, :(n + self.bs - 1) // self.bs].tolist()) for b, n in enumerate(lens)]
        free = self.stack[:int(self.free)].cpu().tolist()
        everything = free + [i for u in used for i in u]
        assert sorted(everything) == list(range(self.kc.shape[1]))  # no block lost, none held twice


STEPS = [[16, 3, 0, 17, 1], [7, 30, 16, 1, 1], [1, -1, 40, 16, 9], [20, 20, 5, -1, 33], [-1, -1, -1, -1, -1], [7, 0, 1, 0, 64],
         [12, 12, 12, 12, 12], [18, 18, 18, 18, 18]]


def test_steps_of_the_operators_together():
    s = Step(1)
    for new in STEPS:
        s.inputs(new)
        s.run()
        s.check()


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
    direct.qw.copy_(a.qw)
    direct.kw.copy_(a.kw)
    for new in STEPS:
        for s, g in zip((a, b), graphs):
            s.inputs(new)
            g.replay()
        direct.inputs(new)
        direct.run()
        a.check()
        b.check()
        t = int(direct.off[-1])
        assert torch.equal(a.out[:, :t], direct.out[:, :t]) and torch.equal(a.lens, direct.lens)
        assert torch.equal(a.kc.view(torch.int16), direct.kc.view(torch.int16)) and torch.equal(a.tables, direct.tables)


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
