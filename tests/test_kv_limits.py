"""Sizes at the ends of what the cache's entry points take, on the CPU: every answer comes before a launch."""
import pytest

import weight_only_quantization_amd as hq
from tests.test_kv_abi import BAD, FAKE, WS, attention, cache, lib  # noqa: F401

MOST = (1 << 31) - (1 << 16) - 1


@pytest.mark.parametrize("past", [1, 1 << 8, 1 << 15, (1 << 16) - 256])
def test_key_counts_near_32_bits(lib, past):  # noqa: F811
    """Kernels look ahead of the last key in 32 bits: lengths that this would carry past 2^31 are refused, the longest
    below them are planned."""
    c = cache(page_size=256)
    one = dict(c=c, total_q=1, num_seqs=1, table_cols=(1 << 23) - 1, table_stride=1 << 23)
    assert attention(lib, max_len=MOST, **one) == WS
    assert attention(lib, max_len=MOST + past, **one) == BAD and "max_len" in hq.last_error()
    e = "hqq_kv_attention_shared"
    assert attention(lib, e, prefix_len=MOST, prefix_table=FAKE, **one) == WS
    assert attention(lib, e, prefix_len=MOST + past, prefix_table=FAKE, **one) == BAD and "prefix_len" in hq.last_error()
