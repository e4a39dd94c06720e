"""GPU: attention of drafted trees in a batch whose slots are mostly without a request, as a step captured at a fixed batch has them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
import tree_reference as ref
from test_gpu_tree_ops import attend_case, check, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device; the CUDA path has no fallback"
    pa.build()
    pa.library()
    yield
    pa.check_error()


class Batch:
    """The requests of a case at these slots of a batch of `slots`; the others are empty."""

    def __init__(self, c, slots, at):
        b, at = len(c["lens"]), np.asarray(at)
        lens, new = np.zeros(slots, np.int32), np.zeros(slots, np.int64)
        tables = np.full((slots, c["tables"].shape[1]), -1, np.int32)
        lens[at], new[at], tables[at] = c["lens"], np.diff(c["off"]), c["tables"]
        assert len(at) == b and (np.diff(at) > 0).all()
        self.args = [c["q"].cuda(), c["kc"].cuda(), c["vc"].cuda(), up(ref.words_of(c["seen"])), up(tables), up(lens),
                     up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))]
        self.out = torch.full_like(self.args[0], 9.0)
        q, k = self.args[0], self.args[1]
        need = pa.attend_tree_workspace_size(q.shape[0], slots, q.shape[1], k.shape[1], k.shape[3], k.shape[2], tables.shape[1], q.dtype)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def run(self):
        return pa.attend_tree(*self.args, out=self.out, workspace=self.ws)


OLD, NEW = [700, 5, 128, 3000, 0, 64], [16, 1, 40, 3, 100, 7]


@pytest.mark.parametrize("slots,at", [
    (6, range(6)), (40, [0, 1, 2, 3, 4, 39]), (100, [31, 32, 63, 64, 65, 98]), (300, [0, 32, 65, 98, 130, 230]), (4096, range(6)),
    (4096, range(4090, 4096)), (8192, [0, 1000, 1001, 1034, 5000, 8191]), (8192, [447, 448, 449, 4000, 4031, 4032])])
def test_empty_slots_change_nothing(slots, at):
    c = attend_case(np.random.default_rng(1), 8, 2, 128, 16, "bf16", OLD, NEW)
    alone, batch = Batch(c, 6, range(6)), Batch(c, slots, at)
    alone.run()
    batch.run()
    pa.check_error()
    check(c, batch.out)
    assert torch.equal(batch.out, alone.out)


@pytest.mark.parametrize("old,new", [([3000], [1]), ([1000] * 32, [16] * 32)])
def test_empty_slots_behind_the_last_request_are_not_walked_one_by_one(old, new):
    """8192 slots take less than five times as long as the active ones alone (passed one after the other, they took 16 and 34 times)."""
    c = attend_case(np.random.default_rng(2), 28, 4, 128, 16, "bf16", old, new)

    def time_of(batch):
        for _ in range(3):
            batch.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                batch.run()
        best = float("inf")
        for _ in range(7):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert time_of(Batch(c, 8192, range(len(old)))) < 5 * time_of(Batch(c, len(old), range(len(old))))
