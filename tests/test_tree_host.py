"""Host-side checks of the operators of a speculative step with a drafted tree (no GPU): argument validation, and the plain
forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
import tree_reference as ref

P = 1 << 30  # an aligned, never-dereferenced address; buffers below are far apart


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.library()


def spaced(n):
    return [P + (i << 44) for i in range(n)]


def check(fn, ok, changes, status):
    for i, value in changes.items():
        args = list(ok)
        args[i] = value
        assert fn(*args) == status, (i, value)


def test_tree_masks_rejects_bad_arguments(lib):
    b = spaced(5)  # positions, mask, parents, lens, offsets
    ok = b + [4, 64, 2, None]
    for i in range(5):
        check(lib.pa_tree_masks, ok, {i: None}, 1)
        check(lib.pa_tree_masks, ok, {i: b[i] + 2}, 1)
    check(lib.pa_tree_masks, ok, {1: b[1] + 4, 5: 8193, 6: -1, 7: 0}, 1)
    check(lib.pa_tree_masks, ok, {5: -1, 6: 0x7FFF0001, 7: 17}, 1)
    check(lib.pa_tree_masks, ok, {0: b[2] + 128, 1: b[0] + 8, 3: b[1] + 1016, 4: b[0] + 252}, 1)
    empty = [None] * 5 + [0, 0, 1, None]
    assert lib.pa_tree_masks(*empty) == 0


def test_accept_tree_rejects_bad_arguments(lib):
    b = spaced(7)  # accepted, number, next, parents, tokens, choices, offsets
    ok = b + [4, 64, 8, 8, None]
    for i in range(7):
        check(lib.pa_accept_tree, ok, {i: None}, 1)
        check(lib.pa_accept_tree, ok, {i: b[i] + 2}, 1)
    check(lib.pa_accept_tree, ok, {2: b[2] + 4, 4: b[4] + 4, 7: 8193, 8: -1, 9: 0, 10: 2}, 1)
    check(lib.pa_accept_tree, ok, {7: -1, 9: 1025, 10: 0}, 1)
    check(lib.pa_accept_tree, ok, {0: b[1] + 8, 1: b[3] + 252, 2: b[5] + 504, 6: b[0] + 124}, 1)
    assert lib.pa_accept_tree(*([None] * 7 + [0, 0, 1, 4, None])) == 0


def test_compact_tree_rejects_bad_arguments(lib):
    arr = ctypes.c_void_p * 2
    keys, values = arr(P + (40 << 44), P + (41 << 44)), arr(P + (42 << 44), P + (43 << 44))
    b = spaced(10)  # slots, offsets, accepted, number, tables, lens, stack, count, lens out, count out
    ok = [keys, values, 2] + b + [4, 64, 5, 2, 128, 16, 8, 100, 2, None]
    for i in range(3, 13):
        check(lib.pa_compact_tree, ok, {i: None}, 1)
        check(lib.pa_compact_tree, ok, {i: ok[i] + 2}, 1)
    check(lib.pa_compact_tree, ok, {0: None, 1: None, 2: 0}, 1)
    check(lib.pa_compact_tree, ok, {2: 257, 13: 8193, 14: -1, 15: 0, 16: 0, 17: 0, 18: 0, 19: 0, 20: 0, 21: 3}, 1)
    check(lib.pa_compact_tree, ok, {13: -1, 15: 1025, 19: 1 << 28, 20: 0x7FFF0001, 21: -1}, 1)
    check(lib.pa_compact_tree, ok, {0: arr(P, None), 1: arr(P + 1, P)}, 1)
    # overlaps: lengths and count alone may be in place
    check(lib.pa_compact_tree, ok, {9: b[4], 11: b[3], 12: b[1] + 16, 10: b[8] + 4, 8: b[6] + 96}, 1)
    check(lib.pa_compact_tree, ok, {11: b[5] + 4, 12: b[8] + 12}, 1)


def test_norm_rope_write_rejects_bad_arguments(lib):
    b = spaced(11)  # query_out, query, key, value, key_cache, value_cache, q_weight, k_weight, inv_freq, positions, slots
    ok = b + [512, 256, 256, 8, 4, 2, 128, 128, 0, 1.0, 1e-6, 0.0, 0, 16, 10, 2, None]
    for i in (0, 1, 2, 3, 4, 5, 8, 9, 10):
        check(lib.pa_norm_rope_write_kv, ok, {i: None}, 1)
    for i in range(11):
        check(lib.pa_norm_rope_write_kv, ok, {i: b[i] + 1}, 1)
    check(lib.pa_norm_rope_write_kv, ok, {11: 511, 12: 255, 13: 255, 14: -1, 15: 0, 16: 0, 17: 127, 18: 130, 19: 2}, 1)
    check(lib.pa_norm_rope_write_kv, ok, {14: 0x7FFF0001, 18: 63, 20: float("nan"), 21: -1e-6, 22: float("inf"), 23: 3}, 1)
    check(lib.pa_norm_rope_write_kv, ok, {21: float("nan"), 24: 0, 25: 0, 26: 3}, 1)
    check(lib.pa_norm_rope_write_kv, ok, {0: b[1] + 64, 1: b[0] - 64, 2: b[0] + 128, 3: b[0] - 2}, 1)
    wide = list(ok)
    wide[11:14], wide[17] = [2 * 1024, 1024, 1024], 514
    wide[15], wide[16], wide[18] = 2, 1, 514
    assert lib.pa_norm_rope_write_kv(*wide) == 2
    assert lib.pa_norm_rope_write_kv(*([None] * 11 + [512, 256, 256, 0, 4, 2, 128, 0, 0, 1.0, 0.0, 0.0, 0, 16, 10, 2, None])) == 0


def test_attend_tree_rejects_bad_arguments(lib):
    b = spaced(8)  # out, query, key_cache, value_cache, mask, tables, lens, offsets
    ok = b + [4, 64, 8, 2, 128, 16, 8, 100, 1, 0.1, 2, P + (60 << 44), 1 << 40, None]
    for i in range(8):
        check(lib.pa_attend_tree, ok, {i: None}, 1)
        check(lib.pa_attend_tree, ok, {i: b[i] + 2}, 1)
    check(lib.pa_attend_tree, ok, {0: b[0] + 8, 1: b[1] + 8, 2: b[2] + 8, 3: b[3] + 8, 4: b[4] + 4}, 1)
    check(lib.pa_attend_tree, ok, {8: -1, 9: -1, 10: 0, 11: 0, 14: 0, 15: 0, 16: 0, 17: float("nan")}, 1)
    check(lib.pa_attend_tree, ok, {10: 7, 14: 1 << 28, 15: 1 << 27, 9: 1 << 28, 16: 17}, 1)
    check(lib.pa_attend_tree, ok, {8: 8193, 12: 80, 13: 8, 18: 0}, 2)
    check(lib.pa_attend_tree, ok, {12: 256, 13: 64, 18: 3}, 2)
    # out over the query, the caches, the mask, tables, lengths, offsets
    check(lib.pa_attend_tree, ok, {0: b[1] + 64, 1: b[0], 2: b[0] + 1024, 3: b[0], 4: b[0] + 16, 5: b[0], 6: b[0], 7: b[0]}, 1)
    assert lib.pa_attend_tree(*([None] * 8 + [0, 0, 8, 2, 128, 16, 8, 100, 1, 0.1, 2, None, 0, None])) == 0
    assert lib.pa_attend_tree_workspace_size(64, 4, 8, 3, 128, 16, 8, 2) == 0
    assert lib.pa_attend_tree_workspace_size(64, 4, 8, 2, 80, 16, 8, 2) == 0
    assert lib.pa_attend_tree_workspace_size(64, 4, 8, 2, 128, 16, 8, 0) == 0


def test_python_calls_refuse_host_tensors_and_wrong_shapes():
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.tree_masks(i32, i32, i32, 1)
    with pytest.raises(ValueError, match="CUDA"):
        pa.accept_tree(i32, i32, i32, i32, 4)
    x = torch.zeros(2, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pa.attend_tree(x, x, x, i32, i32, i32, i32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.norm_rope_write_kv(x, x, x, x, x, None, None, None, i32, i32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.compact_tree([x], [x], i32, i32, i32, i32, i32, i32, i32, i32)


def test_reference_masks_of_a_small_tree():
    #     0 - 1 - 3
    #      \ 2 - 4    5 a root of its own
    off, parents = np.array([0, 6]), np.array([-1, 0, 0, 1, 2, -1])
    pos, seen = ref.masks(off, parents, [16], 1, 7)
    assert pos.tolist() == [10, 11, 11, 12, 12, 10, 0]
    assert [np.flatnonzero(r).tolist() for r in seen] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [5], []]
    assert ref.words_of(seen)[:, 0].tolist() == [1, 3, 5, 11, 21, 32, 0]


def test_reference_chain_is_causal_attention():
    """The attention of a chain is that of its positions one after the other."""
    rng = np.random.default_rng(3)
    kc, vc, tables, lens = ref.paged(rng, [23], 1, 64, 16, torch.float32)
    kc, vc = kc.double().numpy(), vc.double().numpy()
    off, parents = ref.trees(rng, [7], "chain")
    _, seen = ref.masks(off, parents, lens, 1, 7)
    q = rng.standard_normal((7, 2, 64))
    out, _ = ref.attend(q, kc, vc, tables, lens, off, seen, 0.125, torch.float32)
    flat_k, flat_v = (c[tables[0, :2], 0].reshape(-1, 64) for c in (kc, vc))
    for t in range(7):
        s = 0.125 * q[t] @ flat_k[:17 + t].T
        p = np.exp(s - s.max(1, keepdims=True))
        assert np.allclose(out[t], p / p.sum(1, keepdims=True) @ flat_v[:17 + t], atol=1e-12)
