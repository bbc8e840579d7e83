"""Sizes at the ends of what the cache's entry points take, on the CPU: every answer comes before a launch."""
import pytest

import weight_only_quantization_amd as hq
from tests.test_kv_abi import BAD, FAKE, UNSUP, WS, attention, cache, lib, read, write  # noqa: F401

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


def test_work_past_64_bits(lib):  # noqa: F811
    """KV heads x sequences x row tiles x units of keys whose product wraps to a small number: refused, as the same
    with fewer keys is."""
    kw = dict(c=cache(num_kv_heads=4096, page_size=256), num_q_heads=4096, total_q=1 << 24, num_seqs=32768, cu_q=FAKE,
              table_cols=1 << 22, table_stride=1 << 22)
    for max_q, keys in ((1 << 23, 1 << 12), (1 << 23, ((1 << 22) - 4) * 128), (1 << 23, ((1 << 22) - 3) * 128)):
        # 2^15 row tiles, 2^27 pairs of a head and a sequence, 2^22 units: 2^64
        assert attention(lib, max_q=max_q, max_len=keys, **kw) == UNSUP, keys


def test_launches_past_32_bits(lib):  # noqa: F811
    """Calls with a launch of 2^32 threads or more in a dimension: refused before any kernel of the call runs."""
    for call in (write, read):
        assert call(lib, n=(1 << 28) - 4) == UNSUP and "tokens" in hq.last_error()              # 2 heads of 16 octets: 2^33
        assert call(lib, n=1 << 28, c=cache(head_dim=64, num_kv_heads=2)) == UNSUP
    many = dict(c=cache(num_kv_heads=1024), num_q_heads=1024, total_q=16384, num_seqs=16384, max_len=128)
    assert attention(lib, **many) == UNSUP and "sequences" in hq.last_error()                   # 2^24 blocks
    e = "hqq_kv_attention_shared"
    rows = dict(num_q_heads=64, c=cache(num_kv_heads=64), total_q=1 << 20, num_seqs=1 << 10, max_len=128, prefix_table=FAKE)
    assert attention(lib, e, prefix_len=128, **rows) == UNSUP and "query rows" in hq.last_error()  # a join of 2^26 rows
    rows["total_q"] -= 1 << 10
    assert attention(lib, e, prefix_len=128, **rows) == WS


@pytest.mark.parametrize("name", ["seq_lens", "page_table", "cu_q", "prefix_table", "lse"])
def test_misaligned_words(lib, name):  # noqa: F811
    """Lists of 32-bit words off their alignment: scalar loads would read others in their place."""
    kw = dict(max_len=128, cu_q=FAKE, max_q=2, prefix_table=FAKE, prefix_len=64, lse=FAKE)
    assert attention(lib, "hqq_kv_attention_shared", **kw) == WS
    for off in (1, 2, 3):
        kw[name] = FAKE + off
        assert attention(lib, "hqq_kv_attention_shared", **kw) == BAD and "aligned" in hq.last_error()
