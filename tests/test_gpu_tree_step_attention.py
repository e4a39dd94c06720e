"""GPU: attention inside whole steps of drafted trees, against the caches as they were when it read them and within its own bound: a
mask that shows a row one node more or less is seen at once."""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
import tree_reference as ref
from test_gpu_tree_ops import STEPS, Step, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device; the CUDA path has no fallback"
    pa.build()
    pa.library()
    yield
    pa.check_error()


class Kept(Step):
    """A step that keeps its caches as they are between the attention and the compaction."""

    def __init__(self, *args, **more):
        super().__init__(*args, **more)
        self.kept = torch.empty_like(self.kc), torch.empty_like(self.vc)
        self.rows_told = self.rows_seen = 0

    def run(self, stream=None):
        compact = pa.compact_tree

        def keep(*args, **more):
            with torch.cuda.stream(stream):
                for to, cache in zip(self.kept, (self.kc, self.vc)):
                    to.copy_(cache)
            return compact(*args, **more)

        pa.compact_tree = keep
        try:
            super().run(stream)
        finally:
            pa.compact_tree = compact

    def check(self):
        cached = np.array([len(h) for h in self.held])
        cached[self.sizes < 0] = 0
        lens = cached + np.maximum(self.sizes, 0)
        _, seen = ref.masks(self.off, self.host_parents, lens, 1, self.rows)
        t, tables = int(self.off[-1]), self.tables.cpu().numpy()
        got, q, kc, vc = (f64(x) for x in (self.out, self.turned, *self.kept))
        less, more = seen.copy(), seen.copy()  # masks with mistakes: without the node itself, and with all nodes of its request
        for b in range(self.b):
            n = int(self.off[b + 1] - self.off[b])
            less[np.arange(self.off[b], self.off[b + 1]), np.arange(n)] = False
            more[self.off[b]:self.off[b + 1], :n] = True
        for l in range(self.layers):
            args = (q[l], kc[l], vc[l], tables, lens, self.off)
            want, bound = ref.attend(*args, seen, self.d ** -0.5, torch.bfloat16)
            assert (np.abs(got[l][:t] - want[:t]) <= bound[:t]).all()
            for wrong in (less, more):
                differs = np.flatnonzero((wrong[:t] != seen[:t]).any(1))
                other, _ = ref.attend(*args, wrong, self.d ** -0.5, torch.bfloat16)
                self.rows_seen += len(differs)
                self.rows_told += int((np.abs(got[l][differs] - other[differs]) > bound[differs]).any((1, 2)).sum())
        super().check()


def test_attention_of_steps_reads_what_it_should():
    s = Kept(11, width=40)
    for new in STEPS + [[50, 7, 30, 1, 5]] * 4:  # (the last ones on contexts of some hundred positions)
        s.inputs(new)
        s.run()
        s.check()
    assert s.rows_told > 0.99 * s.rows_seen > 1000  # the bound tells a mask with a mistake from the right one


def test_attention_of_captured_steps_and_of_two_streams_reads_what_it_should():
    a, b = Kept(12), Kept(13)
    a.inputs([0] * 5)
    a.run()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        a.run(stream=torch.cuda.current_stream())
    for new in STEPS:
        for s in (a, b):
            s.inputs(new)
        torch.cuda.synchronize()
        graph.replay()
        b.run(stream=stream)
        torch.cuda.synchronize()
        for s in (a, b):
            s.check()
