"""GPU: what the compaction of drafted trees refuses it leaves whole: no row of a request that keeps its length moves, so that
the call can be repeated once its arguments are right."""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
import tree_reference as ref
from test_gpu_tree_ops import compact, compact_case, f64, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device; the CUDA path has no fallback"
    pa.build()
    pa.library()
    yield
    pa.check_error()


def wanted(c, served):
    """The caches, lengths, stack and count when the requests of `served` are compacted and the others left."""
    k, v = f64(c["keys"]), f64(c["values"])
    off, lens, stack, free = c["off"], c["lens"].copy(), c["stack"].copy(), c["free"]
    for b in served:
        one = [off[b:b + 2], c["accepted"][b:b + 1], c["count"][b:b + 1], c["tables"][b:b + 1], lens[b:b + 1]]
        lens[b:b + 1], stack, free = ref.compact([k, v], c["slots"], *one, stack, free, c["bs"])
    return k, v, lens, stack, free


def compare(c, served, keys, values, state, stack):
    k, v, lens, want_stack, free = wanted(c, served)
    assert np.array_equal(f64(keys), k) and np.array_equal(f64(values), v)
    assert state.context_lens.cpu().tolist() == lens.tolist() and int(state.num_free) == free
    if free == c["free"]:
        assert np.array_equal(stack.cpu().numpy(), c["stack"])
    else:
        assert np.array_equal(stack.cpu().numpy()[:free], want_stack[:free])


def two_requests(what):
    """(inputs, the error, the requests that are served, what is put right for another call)."""
    c = compact_case(np.random.default_rng(4), 2, 2, 16, 16, "bf16", [20, 30], [30, 40], 4)
    c["accepted"][:], c["count"][:] = [[0, 2, 4, 20], [0, 1, 7, 39]], 4
    if what == "short":
        right, c["lens"] = {"lens": c["lens"]}, np.array([29, 70], np.int32)
    elif what == "wide":
        right, c["lens"] = {"lens": c["lens"]}, np.array([c["tables"].shape[1] * 16 + 1, 70], np.int32)
    elif what in ("table", "table_low"):
        right = {"tables": c["tables"].copy()}
        c["tables"][0, 3] = len(c["stack"]) if what == "table" else -1
    else:
        right, c["free"] = {"free": c["free"]}, {"room": len(c["stack"]), "count": -1}[what]
    return c, {"short": 7, "wide": 7}.get(what, 5), [] if what in ("room", "count") else [1], right


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what", ["short", "wide", "table", "table_low", "room", "count"])
def test_nothing_of_a_refused_request_moves(what, in_place):
    c, code, served, right = two_requests(what)
    keys, values = c["keys"].cuda(), c["values"].cuda()
    got = []
    assert status(lambda: got.append(compact(c, keys, values, in_place))) == code
    compare(c, served, keys, values, *got[0])
    # put right, the call gives what it would have given at first: for the request that was refused
    c.update(right)
    if served:
        c["count"][1], c["lens"][1] = 0, 70
        c["off"] = np.array([0, 30, 30], np.int32)
    c["keys"], c["values"] = keys.cpu(), values.cpu()
    state, stack = compact(c, keys, values, in_place)
    pa.check_error()
    compare(c, [0, 1], keys, values, state, stack)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests", [3, 300])
@pytest.mark.parametrize("over", [0, 1])
def test_a_stack_with_just_enough_room(requests, over, in_place):
    """A count that leaves room for exactly what is given back, and one more: all requests are served, or none."""
    rng = np.random.default_rng(requests)
    c = compact_case(rng, 2, 1, 8, 16, "f16", rng.integers(0, 60, requests).tolist(), rng.integers(0, 70, requests).tolist(), 12)
    # a fourth of the requests is refused for its path: those give nothing back
    for b in range(0, requests, 4):
        c["count"][b] = 13
    served = [b for b in range(requests) if b % 4]
    given = wanted(c, served)[4] - c["free"]
    bound = sum(-(-int(n) // 16) for n in np.diff(c["off"]))
    assert 0 < given < bound
    c["free"] = len(c["stack"]) - given + over
    c["stack"][:c["free"]] = 5
    keys, values = c["keys"].cuda(), c["values"].cuda()
    got = []
    assert status(lambda: got.append(compact(c, keys, values, in_place))) == (5 if over else 7)
    compare(c, [] if over else served, keys, values, *got[0])


def test_more_blocks_given_back_than_31_bits_count():
    """Offsets that descend between runs that overlap: 2048 requests give back 2^20 blocks each, 2^31 in all, on a stack with room for 8."""
    run, requests = 1 << 20, 4095
    i32 = {"dtype": torch.int32, "device": "cuda"}
    off = torch.tensor([0, run], **i32).repeat(requests // 2 + 1)
    tables = torch.zeros(requests, run, **i32)
    lens = torch.full((requests,), run, **i32)
    around = torch.full((24,), 7, **i32)
    keys, values = (torch.zeros(8, 1, 1, 4, device="cuda") for _ in range(2))
    got = []
    assert status(lambda: got.append(pa.compact_tree(
        [keys], [values], torch.zeros(run, dtype=torch.int64, device="cuda"), off, torch.zeros(requests, 1, **i32), torch.zeros(requests, **i32),
        tables, lens, around[8:16], torch.zeros(1, **i32)))) == 5
    assert torch.equal(got[0].context_lens, lens) and int(got[0].num_free) == 0
    assert (around == 7).all()
