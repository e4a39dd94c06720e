"""Host-side refusals of the serving-step operators at the ends of their sizes (no GPU)."""
import pytest

import paged_kv_cache_129_gb300 as pa

P = 1 << 30  # an aligned, never-dereferenced address
MOST = 0x7FFF0000


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.library()


def far(n):
    """Buffers further apart than any of them is long."""
    return [P + (i << 44) for i in range(n)]


@pytest.mark.parametrize("index", [12, 14])  # blocks, tokens
def test_advance_tables_refuses_counts_next_to_the_end_of_int32(lib, index):
    for count in (MOST + 1, 2 ** 31 - 1):
        args = far(10) + [4, 8, 100, 16, 64, None]
        args[index] = count
        assert lib.pa_advance_tables(*args) == 1 and b"num_tokens" in lib.pa_last_error_string()


def test_rotary_calls_refuse_counts_next_to_the_end_of_int32(lib):
    for count in (MOST + 1, 2 ** 31 - 1):
        write = far(9) + [2, 2, 2, count, 1, 1, 2, 2, 0, 1.0, 16, 10, 2, None]
        assert lib.pa_rope_write_kv(*write) == 1 and b"num_tokens" in lib.pa_last_error_string()
        append = far(12) + [64, 64, 64, 3, count, 1, 1, 64, 64, 0, 1.0, 16, 8, 10, 2, None]
        assert lib.pa_rope_append_fp8(*append) == 1 and b"num_tokens" in lib.pa_last_error_string()
