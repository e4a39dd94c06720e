"""Host-side checks of the caches that the compaction of drafted trees is given (no GPU): none may be listed twice or overlap another,
since each is compacted once per entry, by threads that do not wait for one another."""
import ctypes

import pytest

import paged_kv_cache_129_gb300 as pa

P = 1 << 30  # an aligned, never-dereferenced address; buffers below are far apart
POOL = 100 * 2 * 16 * 128 * 2  # bytes of a cache


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.library()


@pytest.mark.parametrize("layers,change", [
    (2, {"keys": {1: 0}}), (2, {"values": {0: 1}}), (28, {"keys": {27: 3}}), (256, {"values": {255: 0}}),  # a layer's cache again
    (1, {"shared": (0, 0)}), (28, {"shared": (5, 20)}),  # keys that are values
    (2, {"shift": ("keys", 1, 0, POOL - 16)}), (28, {"shift": ("values", 9, 2, -16)}),  # parts of one
])
def test_compact_tree_refuses_caches_that_overlap(lib, layers, change):
    at = {"keys": [P + ((100 + l) << 36) for l in range(layers)], "values": [P + ((500 + l) << 36) for l in range(layers)]}
    for name in ("keys", "values"):
        for to, of in change.get(name, {}).items():
            at[name][to] = at[name][of]
    if "shared" in change:
        at["values"][change["shared"][1]] = at["keys"][change["shared"][0]]
    if "shift" in change:
        name, to, of, by = change["shift"]
        at[name][to] = at[name][of] + by
    arr = ctypes.c_void_p * layers
    b = [P + ((1000 + i) << 36) for i in range(10)]  # slots, offsets, accepted, number, tables, lens, stack, count, lens out, count out
    assert lib.pa_compact_tree(arr(*at["keys"]), arr(*at["values"]), layers, *b, 4, 64, 5, 2, 128, 16, 8, 100, 2, None) == 1
    assert b"overlap" in lib.pa_last_error_string()
