"""GPU: the weights of a node's attention sum to one as they are multiplied: a row over equal values returns that value, as the decode calls do."""
import numpy as np
import pytest
import torch

import paged_kv_cache_129_gb300 as pa
from test_gpu_tree_ops import T, attend, attend_case, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device; the CUDA path has no fallback"
    pa.build()
    pa.library()
    yield
    pa.check_error()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs,old,new", [
    (4, 2, 128, 16, [3, 40, 0], [1, 2, 3]), (28, 4, 128, 16, [700, 1000, 128], [16, 16, 16]), (8, 8, 64, 32, [100, 33, 1], [32, 31, 200]),
    (8, 1, 128, 32, [300, 0, 20], [70, 129, 2]), (4, 4, 64, 16, [5000, 900], [3, 1])])
def test_rows_over_equal_values_return_them(dtype, hq, hkv, d, bs, old, new):
    """Weights and their sum carry the same roundings, and float32 sums of L terms are off by (L / 16 + 16) 2^-23 at most (numerator and
    denominator: 8e-5 at 5003 positions), below the 2^-12 (f16; bf16 2^-9) that would leave a value of the type for its neighbour."""
    c = attend_case(np.random.default_rng(d + bs), hq, hkv, d, bs, dtype, old, new)
    values = torch.from_numpy(np.random.default_rng(7).uniform(0.5, 2.0, (hkv, d)).astype(np.float32)).to(T[dtype])
    c["vc"] = torch.where(c["vc"].isnan(), c["vc"], values[None, :, None, :])
    # scores that grow along the context, so that the weights' reference is often one of an earlier position
    for b, n in enumerate(c["lens"]):
        pos = np.arange(n)
        at = (c["tables"][b, pos // bs], slice(None), pos % bs)
        c["kc"][at] = (c["kc"][at].float() * torch.linspace(0.5, 2.5, int(n))[:, None, None]).to(T[dtype])
    got = f64(attend(c))[:int(c["off"][-1])].reshape(-1, hkv, hq // hkv, d)
    pa.check_error()
    assert np.array_equal(got, np.broadcast_to(f64(values)[None, :, None, :], got.shape))
